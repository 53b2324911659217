// gqa_attn.cu -- attention of new tokens over paged KV8 keys and values with grouped
// query heads: a decode step, a window of speculative tokens, a prompt's chunk
// (causal), or decoder tokens over an encoder's states (unmasked).
//
//   z_t = sm s_k(t) (q . c_k(t)),  out = sum_t softmax(z)_t s_v(t) c_v(t),
// c_k, c_v the e4m3 codes of row t, s_k, s_v its scales.
//
// What bounds it: a decode step reads every row once, 2 D + 8 bytes per row and kv
// head, for G vectors; the products are 8 or 16 vectors wide.  So a row goes straight from
// global memory into the registers of the warp that needs it, as the A operand of a
// 16 x 8 x 16 product (16 rows, or 16 dims, by 8 vectors): no shared memory, no barrier inside
// a tile.
//   * The dims of a score are summed, so their order is free: lane (g, c) of a warp
//     takes 16 bytes at a time of rows g and g + 8, and the queries lie in the same order.  A
//     word of 4 codes is half an operand after two conversions (e4m3 to f16 is exact).
//   * The context's operand pairs rows at one dim: a lane holds the same 16 dims of
//     4 rows and two byte permutes a word pair them up, before the conversion.
//   * The weights come out of the score's accumulators as 8 x 8 blocks of (row, vector)
//     and go into the next product as (vector, row): one transposing move a block.
// A warp takes 16 rows at a time (a page holds at least 16, so they have one page
// entry) and keeps its own running maximum, sum and context; the 4 warps of a CTA
// take turns over the rows and are joined at the tile's end.  32 bf16 sequences of 1k to 65k rows,
// 8 kv heads of 128: 424 us, 5.8 TB/s; 4 of 32768 rows, 2 of 256: 40 us in a row of calls, of which
// 25 are the rows and the rest the walk's start (4,500 cycles), the first loads and the join;
// one of 300 rows 9.7 us, latencies alone.  With vectors on the 16 side of the product, half of
// it empty at 8 vectors, a step took 750 instructions a warp at D = 256 and 255 registers.
//
// Numbers.  Queries are scaled by a power of two to a maximum in [2^14, 2^15) and held
// in f16: bf16 queries exactly (elements below 2^-31 of the largest lose bits), f32
// queries in two halves, to 2^-22.  The running maximum m moves only when a score
// passes it by 2^8.  A context weight is w = p s_v f, p = 2^(z - m), with f per vector so
// that the largest w so far lies in [2^14, 2^16), and goes in two f16 halves: to 2^-22
// of itself or 2^-25 absolute, 2^-39 of the largest, whatever the spread of scales and scores; a million
// such roundings add up to 2^-19.  (f is at most 2^100, also while only rows of zero values have weighed:
// it serves value scales from some 2^-86 on.)  The products' f32 accumulators lose up to
// 2^-23 a step towards zero, so every 32 steps they are added to totals in shared
// memory, and sums of p likewise.
//
// A row that is no number (a NaN code, a scale that is none) makes NaN the vectors that
// see it and no other: in steps that some vector sees only in part, values' NaN codes
// are replaced and flagged, and hidden weights are set to zero rather than multiplied.
#include "gqa_common.cuh"

#include <algorithm>

namespace kvq {
namespace {

using tc::ex2;

constexpr int kNT = 128, kWarps = kNT / 32, kN = 16 * kWarps;
constexpr int kFlush = 32;          // steps between additions to the totals
constexpr int kOv = 1;              // prologue allowance, in steps
// NV blocks of 8 vectors a tile
template <int NV>
using Walk = GqaWalk<8 * NV, kN, kOv, 1>;

template <int D, int NV>
constexpr int sm_ctas() {   // CTAs an SM holds (registers)
    return D * NV >= 512 ? 2 : D * NV >= 256 ? 3 : D * NV == 128 ? 4 : 5;
}

template <int D, int NV, int QP>
struct Smem {
    float4 tot[kWarps][NV][D / 16][32];   // totals of the context, in the accumulators' order
    uint4 q[QP][NV][D / 32][32];          // queries, in operand order, two products' each
    float qs[8 * NV];                     // sm log2(e) 2^e of each vector
    float m[kWarps][8 * NV], l[kWarps][8 * NV], f[kWarps][8 * NV];
    int64_t part[2 * kWarps + 2];
    Walk<NV> walk;
    GqaSegment seg;
    int more;
};

__device__ __forceinline__ void mma16816(float4& d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d.x), "+f"(d.y), "+f"(d.z), "+f"(d.w)
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// Codes are read once by one warp: past L1.
__device__ __forceinline__ uint2 ldg8(const void* p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

template <int D>
struct Rows {   // 16 rows of keys and values, as a lane holds them
    uint32_t k[2][D / 16];   // row 8 t + g, word s: dims 64 (s / 4) + 16 c + 4 (s % 4) ..
    uint32_t v[4][D / 32];   // rows 2 c, 2 c + 1, 2 c + 8, 2 c + 9; word w: dims value_dim(w, g) ..
    float2 s[2];             // scales (key, value) of rows g, g + 8
};
// First dim of word w of the lanes with g.
template <int D>
__device__ __forceinline__ int value_dim(int w, int g) {
    constexpr int kW = D >= 128 ? 4 : 2;   // words of one load
    return 4 * kW * (g + 8 * (w / kW)) + 4 * (w % kW);
}

template <int D>
__device__ __forceinline__ void load_keys(Rows<D>& r, const uint8_t* k, int g, int c) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            const uint4 x = ldg16(k + (8 * t + g) * D + 64 * i + 16 * c);
            r.k[t][4 * i] = x.x;
            r.k[t][4 * i + 1] = x.y;
            r.k[t][4 * i + 2] = x.z;
            r.k[t][4 * i + 3] = x.w;
        }
}
template <int D>
__device__ __forceinline__ void load_values(Rows<D>& r, const uint8_t* v, int g, int c) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint8_t* row = v + (2 * c + (k & 1) + 8 * (k >> 1)) * D;
        if constexpr (D >= 128) {
#pragma unroll
            for (int i = 0; i < D / 128; ++i) {
                const uint4 x = ldg16(row + 16 * (g + 8 * i));
                r.v[k][4 * i] = x.x;
                r.v[k][4 * i + 1] = x.y;
                r.v[k][4 * i + 2] = x.z;
                r.v[k][4 * i + 3] = x.w;
            }
        } else {
            const uint2 x = ldg8(row + 8 * g);
            r.v[k][0] = x.x;
            r.v[k][1] = x.y;
        }
    }
}
template <int D>
__device__ __forceinline__ void load_scales(Rows<D>& r, const float2* s, int g) {
    r.s[0] = s[g];
    r.s[1] = s[g + 8];
}

// Queries of the tile into operand order, kNT / (8 NV) threads a vector.
template <int D, int NV, int QP, typename QT>
__device__ __forceinline__ void load_queries(const GqaParams& p, const GqaSegment& g, Smem<D, NV, QP>& sm) {
    constexpr int kT = kNT / (8 * NV), E = D / kT;
    const int r = threadIdx.x / kT, t = threadIdx.x % kT;
    float x[E];
    const bool live = r < g.vecs;
    const QT* src = static_cast<const QT*>(p.q) + (live ? gqa_vector<D>(p, g, g.vec0 + r) : 0) + t * E;
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        x[i] = live ? (float)src[i] : 0.0f;
        amax = fmaxf(amax, fabsf(x[i]));
    }
#pragma unroll
    for (int o = kT / 2; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
    const int e = max((int)(__float_as_uint(amax) >> 23) - 127 - 14, -110);
    const float up = __uint_as_float((uint32_t)(127 - e) << 23);
    if (t == 0) sm.qs[r] = query_scale(p.sm_scale, e, amax);
#pragma unroll
    for (int i = 0; i < E; i += 2) {
        // word (d % 4) / 2 of product s = 4 (d / 64) + (d % 16) / 4, lane (r % 8, (d % 64) / 16)
        const int d = t * E + i, s = 4 * (d / 64) + (d % 16) / 4, c = (d % 64) / 16, word = 2 * (s & 1) + (d & 3) / 2;
        const float a = x[i] * up, b = x[i + 1] * up;
        const uint32_t hi = pack_half2(a, b);
        reinterpret_cast<uint32_t*>(&sm.q[0][r / 8][s / 2][(r & 7) * 4 + c])[word] = hi;
        if constexpr (QP == 2) {
            const float2 h = unpack_half2(hi);
            reinterpret_cast<uint32_t*>(&sm.q[1][r / 8][s / 2][(r & 7) * 4 + c])[word] = pack_half2(a - h.x, b - h.y);
        }
    }
}

template <typename QT>
__device__ __forceinline__ void store4(QT* dst, float4 v) {
    if constexpr (sizeof(QT) == 4) {
        *reinterpret_cast<float4*>(dst) = v;
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
}

// A lane's accumulators of word w to the output: o[e] = (dim 2 e, vectors 2c, 2c + 1), (dim 2 e + 1, the same).
template <int D, typename QT>
__device__ __forceinline__ void write_out(const GqaParams& p, const GqaSegment& seg, int block, int lane, int w,
                                          const float4 (&o)[2], float il0, float il1) {
    const int d = value_dim<D>(w, lane >> 2), v = 8 * block + 2 * (lane & 3);
    QT* out = static_cast<QT*>(p.out);
    if (v < seg.vecs)
        store4(out + gqa_vector<D>(p, seg, seg.vec0 + v) + d,
               make_float4(o[0].x * il0, o[0].z * il0, o[1].x * il0, o[1].z * il0));
    if (v + 1 < seg.vecs)
        store4(out + gqa_vector<D>(p, seg, seg.vec0 + v + 1) + d,
               make_float4(o[0].y * il1, o[0].w * il1, o[1].y * il1, o[1].w * il1));
}
constexpr float kNone = -3.402823466e38f;   // the maximum of no scores
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }   // no row seen: zeros
__device__ __forceinline__ void scale4(float4& v, float a, float b) {
    v.x *= a;
    v.y *= b;
    v.z *= a;
    v.w *= b;
}
__device__ __forceinline__ void add4(float4& v, const float4& u) {
    v.x += u.x;
    v.y += u.y;
    v.z += u.z;
    v.w += u.w;
}
__device__ __forceinline__ void fma4(float4& v, const float4& u, float a, float b) {
    v.x += u.x * a;
    v.y += u.y * b;
    v.z += u.z * a;
    v.w += u.w * b;
}

template <int D, int NV, int QP, typename QT>
__global__ void __launch_bounds__(kNT, sm_ctas<D, NV>()) gqa_attn_kernel(const __grid_constant__ GqaParams p) {
    extern __shared__ __align__(16) unsigned char raw[];
    using W = Walk<NV>;
    constexpr int kM = 8 * NV;
    Smem<D, NV, QP>& sm = *reinterpret_cast<Smem<D, NV, QP>*>(raw);
    grid_dependency_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    if (tid == 0) p.cuts[blockIdx.x].count = 0;
    if (p.n_seq <= W::kFew) {
        if (warp == 0) {
            W walk;
            const bool any = walk.start_few(p, blockIdx.x, gridDim.x);
            if (lane == 0) {
                sm.walk = walk;
                sm.more = any && walk.get(p, sm.seg);
            }
        }
    } else {
        W walk;
        const bool any = walk.template start_many<kNT>(p, blockIdx.x, gridDim.x, sm.part, sm.part + 2 * kWarps);
        if (tid == 0) {
            sm.walk = walk;
            sm.more = any && walk.get(p, sm.seg);
        }
    }
    __syncthreads();
    // the merge comes early only to a short call: its waiting CTAs, and those of the call
    // behind it, would keep this kernel's from starting
    if (!sm.more || sm.walk.per <= 16) launch_dependents();
    if (!sm.more) return;
    const GqaSegment& seg = sm.seg;
    const int32_t in_page = (1 << p.shift) - 1;
    for (;;) {
        load_queries<D, NV, QP, QT>(p, seg, sm);
        const int32_t all = gqa_limit(p, seg, seg.vec0);   // rows that all vectors see
        const int32_t end = min(seg.limit, seg.u1 * kN), seq = seg.b;
        int32_t r = seg.u0 * kN + warp * 16;
        float4 acc[NV][D / 16];
        float m[NV][2], l[NV][2], tl[NV][2], f[NV][2];   // of vectors 2c and 2c + 1 of each block
#pragma unroll
        for (int b = 0; b < NV; ++b) {
#pragma unroll
            for (int t = 0; t < D / 16; ++t) acc[b][t] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[b][i] = kNone;
                l[b][i] = tl[b][i] = f[b][i] = 0.0f;
            }
        }
        bool flushed = false;
        Rows<D> rows;
        int64_t at = 0;
        int32_t page = 0;
        if (r < end) {
            at = (((int64_t)gqa_page(p, seq, r) * p.n_kv + seg.h) << p.shift) + (r & in_page);
            load_keys<D>(rows, p.k_codes + at * D, g, c);
            load_scales<D>(rows, p.scales + at, g);
            load_values<D>(rows, p.v_codes + at * D, g, c);
            if (r + kN < end) page = gqa_page(p, seq, r + kN);
        }
        __syncthreads();   // queries stored
        float qs[NV][2];
#pragma unroll
        for (int b = 0; b < NV; ++b) {
            qs[b][0] = sm.qs[8 * b + 2 * c];
            qs[b][1] = sm.qs[8 * b + 2 * c + 1];
        }
        int steps = 0;
#pragma unroll 1
        for (; r < end; r += kN) {
            const bool more = r + kN < end;
            if (more) at = (((int64_t)page * p.n_kv + seg.h) << p.shift) + ((r + kN) & in_page);
            if (r + 2 * kN < end) page = gqa_page(p, seq, r + 2 * kN);
            // scores: (row g, vectors 2c, 2c + 1), (row g + 8, the same)
            float z[NV][4];
            {
                float4 s4[NV];
#pragma unroll
                for (int b = 0; b < NV; ++b) s4[b] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int s = 0; s < D / 16; s += 2) {
                    uint32_t a[8];
                    e4m3x4_to_half2x2(rows.k[0][s], a[0], a[2]);
                    e4m3x4_to_half2x2(rows.k[1][s], a[1], a[3]);
                    e4m3x4_to_half2x2(rows.k[0][s + 1], a[4], a[6]);
                    e4m3x4_to_half2x2(rows.k[1][s + 1], a[5], a[7]);
#pragma unroll
                    for (int b = 0; b < NV; ++b)
#pragma unroll
                        for (int q = 0; q < QP; ++q) {
                            const uint4 w = sm.q[q][b][s / 2][lane];
                            mma16816(s4[b], a[0], a[1], a[2], a[3], w.x, w.y);
                            mma16816(s4[b], a[4], a[5], a[6], a[7], w.z, w.w);
                        }
                }
                if (more) load_keys<D>(rows, p.k_codes + at * D, g, c);
                const float sk[2] = {key_scale(rows.s[0].x), key_scale(rows.s[1].x)};
#pragma unroll
                for (int b = 0; b < NV; ++b) {
                    z[b][0] = s4[b].x * sk[0] * qs[b][0];
                    z[b][1] = s4[b].y * sk[0] * qs[b][1];
                    z[b][2] = s4[b].z * sk[1] * qs[b][0];
                    z[b][3] = s4[b].w * sk[1] * qs[b][1];
                }
            }
            float sv[2] = {rows.s[0].y, rows.s[1].y};
            if (more) load_scales<D>(rows, p.scales + at, g);
            const bool partly = r + 16 > all;   // some vector sees these rows in part
            uint32_t hidden = 0u;               // bit 4 b + i: score i of block b
            if (partly) {
                unsigned who[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    bool bad = false;
#pragma unroll
                    for (int w = 0; w < D / 32; ++w) {
                        const uint32_t x = rows.v[k][w], nan = (((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
                        bad |= nan != 0u;
                        rows.v[k][w] = x ^ nan;
                    }
                    who[k] = __ballot_sync(kFull, bad);
                }
                // row g lies with the lanes c = g / 2, at place g % 2
                const unsigned lanes = 0x11111111u << (g >> 1);
                if ((g & 1 ? who[1] : who[0]) & lanes) sv[0] = __uint_as_float(0x7fffffffu);
                if ((g & 1 ? who[3] : who[2]) & lanes) sv[1] = __uint_as_float(0x7fffffffu);
#pragma unroll
                for (int b = 0; b < NV; ++b)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int32_t lim = gqa_limit(p, seg, seg.vec0 + min(8 * b + 2 * c + i, seg.vecs - 1));
#pragma unroll
                        for (int t = 0; t < 2; ++t)
                            if (r + 8 * t + g >= lim) {
                                z[b][2 * t + i] = -INFINITY;
                                hidden |= 1u << (4 * b + 2 * t + i);
                            }
                    }
            }
            float pr[NV][4], w[NV][4], over = -INFINITY, most = 0.0f;
#pragma unroll
            for (int b = 0; b < NV; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = z[b][i] - m[b][i & 1];
                    over = fmaxf(over, x);
                    pr[b][i] = ex2(x);
                    w[b][i] = pr[b][i] * sv[i >> 1] * f[b][i & 1];   // s_v f may pass f32 where p is 0
                }
            if (partly) {
#pragma unroll
                for (int b = 0; b < NV; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (hidden & (1u << (4 * b + i))) w[b][i] = 0.0f;
            }
#pragma unroll
            for (int b = 0; b < NV; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) most = fmaxf(most, fabsf(w[b][i]));
            const bool lift = over > 8.0f || most > 60000.0f;
            if (__any_sync(kFull, lift)) {
                // new maxima, new factors f, and what is summed so far brought to them
#pragma unroll
                for (int b = 0; b < NV; ++b) {
                    float k[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float n = fmaxf(m[b][i], fmaxf(z[b][i], z[b][2 + i]));
#pragma unroll
                        for (int o = 4; o <= 16; o <<= 1) n = fmaxf(n, __shfl_xor_sync(kFull, n, o));
                        float top = 0.0f;
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const int j = 2 * t + i;
                            pr[b][j] = ex2(z[b][j] - n);
                            w[b][j] = hidden & (1u << (4 * b + j)) ? 0.0f : pr[b][j] * sv[t];
                            top = fmaxf(top, fabsf(w[b][j]));
                        }
#pragma unroll
                        for (int o = 4; o <= 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
                        const float d = ex2(m[b][i] - n), f0 = f[b][i];
                        // the largest weight so far, at most 2^14 / f, against the step's
                        const float large = fmaxf(top, f0 > 0.0f ? d * 0x1p14f / f0 : 0.0f);
                        // (rows of zero values weigh nothing yet: the largest factor, with which the first
                        // weight passes 60000 and lifts; a factor of 0 would hide all that follow)
                        const float f1 = fminf(0x1p14f / large, 0x1p100f);
                        k[i] = f0 > 0.0f ? d * (f1 / f0) : 0.0f;
                        l[b][i] *= d;
                        tl[b][i] *= d;
                        m[b][i] = n;
                        f[b][i] = f1;
                        w[b][i] *= f1;
                        w[b][2 + i] *= f1;
                    }
#pragma unroll
                    for (int t = 0; t < D / 16; ++t) scale4(acc[b][t], k[0], k[1]);
                    if (flushed) {
#pragma unroll 4
                        for (int t = 0; t < D / 16; ++t) scale4(sm.tot[warp][b][t][lane], k[0], k[1]);
                    }
                }
            }
            // weights as the context's operand: (vector g, rows 2c, 2c + 1) and rows 8 further, two f16 halves
            uint32_t hi[NV][2], lo[NV][2];
#pragma unroll
            for (int b = 0; b < NV; ++b) {
                l[b][0] += pr[b][0] + pr[b][2];
                l[b][1] += pr[b][1] + pr[b][3];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint32_t h = pack_half2(w[b][2 * t], w[b][2 * t + 1]);
                    const float2 x = unpack_half2(h);
                    hi[b][t] = transpose8x8(h);
                    lo[b][t] = transpose8x8(pack_half2(w[b][2 * t] - x.x, w[b][2 * t + 1] - x.y));
                }
            }
#pragma unroll
            for (int wd = 0; wd < D / 32; ++wd) {
                uint32_t x[4], y[4];   // rows 2c, 2c + 1 at dims 0 .. 3 of the word; rows 8 further
                e4m3x4_to_half2x2(__byte_perm(rows.v[0][wd], rows.v[1][wd], 0x5140), x[0], x[1]);
                e4m3x4_to_half2x2(__byte_perm(rows.v[0][wd], rows.v[1][wd], 0x7362), x[2], x[3]);
                e4m3x4_to_half2x2(__byte_perm(rows.v[2][wd], rows.v[3][wd], 0x5140), y[0], y[1]);
                e4m3x4_to_half2x2(__byte_perm(rows.v[2][wd], rows.v[3][wd], 0x7362), y[2], y[3]);
#pragma unroll
                for (int b = 0; b < NV; ++b)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        mma16816(acc[b][2 * wd + e], x[2 * e], x[2 * e + 1], y[2 * e], y[2 * e + 1], hi[b][0], hi[b][1]);
                        mma16816(acc[b][2 * wd + e], x[2 * e], x[2 * e + 1], y[2 * e], y[2 * e + 1], lo[b][0], lo[b][1]);
                    }
            }
            if (more) load_values<D>(rows, p.v_codes + at * D, g, c);
            if (++steps == kFlush) {
                steps = 0;
#pragma unroll
                for (int b = 0; b < NV; ++b) {
#pragma unroll
                    for (int t = 0; t < D / 16; ++t) {
                        if (flushed) add4(acc[b][t], sm.tot[warp][b][t][lane]);
                        sm.tot[warp][b][t][lane] = acc[b][t];
                        acc[b][t] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        tl[b][i] += l[b][i];
                        l[b][i] = 0.0f;
                    }
                }
                flushed = true;
            }
        }
        // the warp's state to shared memory
#pragma unroll
        for (int b = 0; b < NV; ++b) {
#pragma unroll
            for (int t = 0; t < D / 16; ++t) {
                if (flushed) add4(acc[b][t], sm.tot[warp][b][t][lane]);
                sm.tot[warp][b][t][lane] = acc[b][t];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float x = tl[b][i] + l[b][i];
#pragma unroll
                for (int o = 4; o <= 16; o <<= 1) x += __shfl_xor_sync(kFull, x, o);
                if (g == 0) {
                    sm.m[warp][8 * b + 2 * c + i] = m[b][i];
                    sm.l[warp][8 * b + 2 * c + i] = x;
                    sm.f[warp][8 * b + 2 * c + i] = f[b][i];
                }
            }
        }
        __syncthreads();
        // the warps' states joined, a (block, word) a warp at a time
        const bool whole = seg.slot < 0;
        for (int it = warp; it < NV * (D / 32); it += kWarps) {
            const int b = it / (D / 32), wd = it % (D / 32), v0 = 8 * b + 2 * c;
            float top[2] = {kNone, kNone}, sum[2] = {0.0f, 0.0f};
            float4 o[2] = {};
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                top[0] = fmaxf(top[0], sm.m[i][v0]);
                top[1] = fmaxf(top[1], sm.m[i][v0 + 1]);
            }
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                float k[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float x = ex2(sm.m[i][v0 + j] - top[j]), f0 = sm.f[i][v0 + j];
                    sum[j] += sm.l[i][v0 + j] * x;
                    k[j] = f0 > 0.0f ? x / f0 : 0.0f;
                }
                fma4(o[0], sm.tot[i][b][2 * wd][lane], k[0], k[1]);
                fma4(o[1], sm.tot[i][b][2 * wd + 1][lane], k[0], k[1]);
            }
            if (whole) {
                write_out<D, QT>(p, seg, b, lane, wd, o, inverse_sum(sum[0]), inverse_sum(sum[1]));
            } else {
                float4* dst = reinterpret_cast<float4*>(p.ws_o) + ((int64_t)seg.slot * NV * (D / 16) + 2 * it) * 32 + lane;
                dst[0] = o[0];
                dst[32] = o[1];
                if (wd == 0 && g == 0) {
                    p.ws_ml[seg.slot * kM + v0] = make_float2(top[0], sum[0]);
                    p.ws_ml[seg.slot * kM + v0 + 1] = make_float2(top[1], sum[1]);
                }
            }
        }
        // a CTA begins one cut tile at most, its last
        if (tid == 0 && !whole && seg.u0 == 0) p.cuts[blockIdx.x] = GqaCut{seg.count, seg.h, seg.vec0, seg.vecs, seg.q0};
        if (seg.last) break;
        __syncthreads();   // the segment is read
        if (warp == 0) {
            W walk = sm.walk;
            const bool more = walk.next(p);
            __syncwarp();
            if (lane == 0) {
                sm.walk = walk;
                sm.more = more && walk.get(p, sm.seg);
            }
        }
        __syncthreads();   // the totals and queries are free for the next tile
        if (!sm.more) break;
    }
}

// Cut tiles joined, CTA (c, block and word) for the tile that CTA c of the walk began; its
// warps share the tile's states.
constexpr int kMergeNT = 128;
template <int D, int NV, typename QT>
__global__ void __launch_bounds__(kMergeNT) gqa_merge_kernel(const __grid_constant__ GqaParams p) {
    constexpr int kMW = kMergeNT / 32, kM = 8 * NV;
    __shared__ float4 part[kMW][2][32], stat[kMW][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = lane & 3, first = blockIdx.x, sub = blockIdx.y;
    const int b = sub / (D / 32), wd = sub % (D / 32), v0 = 8 * b + 2 * c;
    grid_dependency_wait();
    launch_dependents();
    const GqaCut cut = p.cuts[first];
    if (cut.count == 0) return;
    // (maximum, sum) of vectors 2c and 2c + 1
    float4 st = make_float4(kNone, 0.0f, kNone, 0.0f), o[2] = {};
#pragma unroll 4
    for (int i = warp; i < cut.count; i += kMW) {
        const int sl = Walk<NV>::slot(first + i, first);
        const float4 a = __ldcg(reinterpret_cast<const float4*>(p.ws_ml + sl * kM + v0));
        const float4* src = reinterpret_cast<const float4*>(p.ws_o) + ((int64_t)sl * NV * (D / 16) + 2 * sub) * 32 + lane;
        const float4 x = __ldcg(src), y = __ldcg(src + 32);
        const float n0 = fmaxf(st.x, a.x), n1 = fmaxf(st.z, a.z);
        const float s0 = ex2(st.x - n0), s1 = ex2(st.z - n1), k0 = ex2(a.x - n0), k1 = ex2(a.z - n1);
        st = make_float4(n0, st.y * s0 + a.y * k0, n1, st.w * s1 + a.w * k1);
        scale4(o[0], s0, s1);
        scale4(o[1], s0, s1);
        fma4(o[0], x, k0, k1);
        fma4(o[1], y, k0, k1);
    }
    part[warp][0][lane] = o[0];
    part[warp][1][lane] = o[1];
    stat[warp][lane] = st;
    __syncthreads();
    if (warp != 0) return;
    float top0 = kNone, top1 = kNone, sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
    for (int w = 0; w < kMW; ++w) {
        top0 = fmaxf(top0, stat[w][lane].x);
        top1 = fmaxf(top1, stat[w][lane].z);
    }
    o[0] = o[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kMW; ++w) {
        const float4 a = stat[w][lane];
        const float k0 = ex2(a.x - top0), k1 = ex2(a.z - top1);
        sum0 += a.y * k0;
        sum1 += a.w * k1;
        fma4(o[0], part[w][0][lane], k0, k1);
        fma4(o[1], part[w][1][lane], k0, k1);
    }
    GqaSegment seg;
    seg.h = cut.h;
    seg.vec0 = cut.vec0;
    seg.vecs = cut.vecs;
    seg.q0 = cut.q0;
    write_out<D, QT>(p, seg, b, lane, wd, o, inverse_sum(sum0), inverse_sum(sum1));
}

template <int D, int NV, int QP, typename QT>
cudaError_t launch_kernel(const GqaParams& p, cudaStream_t stream) {
    constexpr size_t smem = sizeof(Smem<D, NV, QP>);
    constexpr int ctas = 152 * sm_ctas<D, NV>();
    static_assert(ctas <= kGqaMaxCtas, "workspace");
    cudaError_t e =
        cudaFuncSetAttribute(gqa_attn_kernel<D, NV, QP, QT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    timing_mark(stream, 0);
    e = launch_chained(gqa_attn_kernel<D, NV, QP, QT>, ctas, kNT, smem, stream, p);
    timing_mark(stream, 1);
    if (e == cudaSuccess)
        e = launch_chained(gqa_merge_kernel<D, NV, QT>, dim3(ctas, NV * (D / 32)), kMergeNT, 0, stream, p);
    timing_mark(stream, 2);
    return e;
}
// Blocks of 8 vectors a tile: one where a sequence's vectors of a kv head fill no more on
// average, else two.
template <int D, int QP, typename QT>
cudaError_t launch_dims(const GqaParams& p, cudaStream_t stream) {
    return p.max_tok * p.group <= 8 * (int64_t)p.n_seq ? launch_kernel<D, 1, QP, QT>(p, stream)
                                                       : launch_kernel<D, 2, QP, QT>(p, stream);
}
template <int D>
cudaError_t launch_type(const GqaParams& p, kvq_dtype dt, cudaStream_t stream) {
    return dt == KVQ_BF16 ? launch_dims<D, 1, __nv_bfloat16>(p, stream) : launch_dims<D, 2, float>(p, stream);
}

// Above so many vectors of a sequence and kv head, on average, the tensor-core kernel takes less
// time (16 sequences of 4000 rows, 8 kv heads of 128, bf16: 16 vectors 72 us against 58, 32
// vectors 72 against 89; f32: 32 vectors 134 against 96, 64 vectors 144 against 164).
constexpr int64_t tensor_vectors(kvq_dtype dt) { return dt == KVQ_BF16 ? 24 : 48; }

}  // namespace

// Error word, the cut tiles, their maxima and sums, their contexts.
size_t gqa_attn_workspace_bytes(int32_t head_dim) {
    const size_t own = (size_t)2 * kGqaMaxCtas * 16 * (sizeof(float2) + head_dim * sizeof(float));
    return kWsHeader + kGqaCutBytes + std::max(own, gqa_tc_state_bytes(head_dim));
}

cudaError_t launch_gqa_attn(const GqaAttnCall& c, cudaStream_t stream) {
    GqaParams p{};
    p.n_seq = c.n_seq;
    p.n_heads = c.n_heads;
    p.n_kv = c.n_kv_heads;
    p.group = c.n_heads / c.n_kv_heads;
    p.causal = c.causal;
    p.q = c.q;
    p.out = c.out;
    p.k_codes = c.k_codes;
    p.v_codes = c.v_codes;
    p.scales = reinterpret_cast<const float2*>(c.scales);
    p.cu_q = c.cu_q;
    p.kv_lens = c.kv_lens;
    p.table = c.table;
    p.table_stride = c.table_stride;
    while ((1 << p.shift) < c.page_rows) ++p.shift;
    p.n_pages = c.n_pages;
    p.max_tok = c.n_tokens;
    p.sm_scale = c.sm_scale;
    char* ws = static_cast<char*>(c.workspace);
    p.err = reinterpret_cast<int32_t*>(ws);
    p.cuts = reinterpret_cast<GqaCut*>(ws + kWsHeader);
    p.ws_ml = reinterpret_cast<float2*>(ws + kWsHeader + kGqaCutBytes);
    p.ws_o = reinterpret_cast<float*>(p.ws_ml + 2 * kGqaMaxCtas * 16);
    if (gqa_tc_supported(c.head_dim, c.dtype) && p.max_tok * p.group > tensor_vectors(c.dtype) * p.n_seq)
        return launch_gqa_tc(p, c.head_dim, c.dtype, p.ws_ml, stream);
    switch (c.head_dim) {
        case 64: return launch_type<64>(p, c.dtype, stream);
        case 128: return launch_type<128>(p, c.dtype, stream);
        case 256: return launch_type<256>(p, c.dtype, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace kvq
