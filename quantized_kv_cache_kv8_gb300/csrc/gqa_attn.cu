// gqa_attn.cu -- attention of new tokens over paged KV8 keys and values with grouped
// query heads: a decode step, a window of speculative tokens, a prompt's chunk
// (causal), or decoder tokens over an encoder's states (unmasked).
//
//   z_t = sm s_k(t) (q . c_k(t)),  out = sum_t softmax(z)_t s_v(t) c_v(t),
// c_k, c_v the e4m3 codes of row t, s_k, s_v its scales.
//
// What bounds it: a decode step reads every row once, 2 D + 8 bytes per row and kv
// head, for G vectors; the products are M = 16 at most.  So a row goes straight from
// global memory into the registers of the warp that needs it, as the operand of a
// 16 x 8 x 16 product: no shared memory, no barrier inside a tile.
//   * The dims of a score are summed, so their order is free: lane (g, c) of a warp
//     takes 16 bytes at a time of row g, and the queries lie in the same order.  A
//     word of 4 codes is one operand after two conversions (e4m3 to f16 is exact).
//   * The value's operand pairs rows at one dim: a lane holds the same 16 dims of
//     4 rows and two byte permutes a word pair them up, before the conversion.
//   * The order of the rows in both is that of the accumulator, so the weights go
//     from the score's accumulators to the next product's operand as they lie.
// A warp takes 16 rows at a time (a page holds at least 16, so they have one page
// entry) and keeps its own running maximum, sum and context; the 4 warps of a CTA
// take turns over the rows and are joined at the tile's end.
//
// Numbers.  Queries are scaled by a power of two to a maximum in [2^14, 2^15) and held
// in f16: bf16 queries exactly (elements below 2^-31 of the largest lose bits), f32
// queries in two halves, to 2^-22.  The running maximum m moves only when a score
// passes it by 2^8.  A context weight is w = p s_v f, p = 2^(z - m), with f per vector so
// that the largest w so far lies in [2^14, 2^16), and goes in two f16 halves: to 2^-22
// of itself or 2^-25 absolute, 2^-39 of the largest, whatever the spread of scales and scores; a million
// such roundings add up to 2^-19.  The products' f32 accumulators lose up to
// 2^-23 a step towards zero, so every 32 steps they are added to totals in shared
// memory, and sums of p likewise.
//
// A row that is no number (a NaN code, a scale that is none) makes NaN the vectors that
// see it and no other: in steps that some vector sees only in part, values' NaN codes
// are replaced and flagged, and hidden weights are set to zero rather than multiplied.
#include "gqa_common.cuh"
#include "tc_common.cuh"

#include <algorithm>

namespace kvq {
namespace {

using tc::ex2;
using tc::kLog2e;

constexpr int kNT = 128, kWarps = kNT / 32, kM = 16, kN = 16 * kWarps;
constexpr int kFlush = 32;          // steps between additions to the totals
constexpr int kOv = 1;              // prologue allowance, in steps
using Walk = GqaWalk<kM, kN, kOv>;

template <int D>
constexpr int sm_ctas() { return D == 256 ? 2 : D == 128 ? 3 : 4; }   // CTAs an SM holds (registers)

template <int D, int QP>
struct Smem {
    float4 tot[kWarps][D / 8][32];   // totals of the context, in the accumulators' order
    uint4 q[QP][D / 16][32];         // queries, in operand order
    float qs[kM];                    // sm log2(e) 2^e of each vector
    float m[kWarps][kM], l[kWarps][kM], f[kWarps][kM];
    int64_t part[kWarps + 10];
    Walk walk;
    GqaSegment seg;
    int more, last;
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }

// Codes are read once by one warp: past L1.
__device__ __forceinline__ uint4 ldg16(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ldg8(const void* p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

template <int D>
struct Rows {   // 16 rows of keys and values, as a lane holds them
    uint32_t k[2][D / 16];   // row 8 t + g, word s: dims 64 (s / 4) + 16 c + 4 (s % 4) ..
    uint32_t v[4][D / 32];   // rows 2 c, 2 c + 1, 2 c + 8, 2 c + 9; word w: dims value_dim(w, g) ..
    float4 s[2];             // scales (k, v) of rows 8 t + 2 c, 8 t + 2 c + 1
};
// First dim of word w of the lanes with g, and of the accumulators of column g.
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
__device__ __forceinline__ void load_scales(Rows<D>& r, const float2* s, int c) {
    r.s[0] = *reinterpret_cast<const float4*>(s + 2 * c);
    r.s[1] = *reinterpret_cast<const float4*>(s + 8 + 2 * c);
}

// Queries of the tile into operand order, 8 threads a vector.
template <int D, int QP, typename QT>
__device__ __forceinline__ void load_queries(const GqaParams& p, const GqaSegment& g, Smem<D, QP>& sm) {
    const int r = threadIdx.x / 8, t = threadIdx.x % 8;
    constexpr int E = D / 8;
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
    for (int o = 4; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
    const int e = max((int)(__float_as_uint(amax) >> 23) - 127 - 14, -110);
    const float up = __uint_as_float((uint32_t)(127 - e) << 23);
    if (t == 0) sm.qs[r] = p.sm_scale * kLog2e * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
    for (int i = 0; i < E; i += 2) {
        const int d = t * E + i, s = 4 * (d / 64) + (d % 16) / 4, c = (d % 64) / 16;
        const float a = x[i] * up, b = x[i + 1] * up;
        const uint32_t hi = pack_half2(a, b);
        const int word = 2 * ((d & 3) / 2) + r / 8;
        reinterpret_cast<uint32_t*>(&sm.q[0][s][(r & 7) * 4 + c])[word] = hi;
        if constexpr (QP == 2) {
            const float2 h = unpack_half2(hi);
            reinterpret_cast<uint32_t*>(&sm.q[1][s][(r & 7) * 4 + c])[word] = pack_half2(a - h.x, b - h.y);
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

// Four accumulator tiles (word w) of a lane to the output: o[e] = columns (g, 2c), (g, 2c+1),
// (g+8, 2c), (g+8, 2c+1) of dim e of the word.
template <int D, typename QT>
__device__ __forceinline__ void write_out(const GqaParams& p, const GqaSegment& seg, int lane, int w, const float4 (&o)[4],
                                          float il0, float il1) {
    const int g = lane >> 2, c = lane & 3;
    QT* out = static_cast<QT*>(p.out);
    if (g < seg.vecs) {
        QT* d = out + gqa_vector<D>(p, seg, seg.vec0 + g);
        store4(d + value_dim<D>(w, 2 * c), make_float4(o[0].x * il0, o[1].x * il0, o[2].x * il0, o[3].x * il0));
        store4(d + value_dim<D>(w, 2 * c + 1), make_float4(o[0].y * il0, o[1].y * il0, o[2].y * il0, o[3].y * il0));
    }
    if (g + 8 < seg.vecs) {
        QT* d = out + gqa_vector<D>(p, seg, seg.vec0 + g + 8);
        store4(d + value_dim<D>(w, 2 * c), make_float4(o[0].z * il1, o[1].z * il1, o[2].z * il1, o[3].z * il1));
        store4(d + value_dim<D>(w, 2 * c + 1), make_float4(o[0].w * il1, o[1].w * il1, o[2].w * il1, o[3].w * il1));
    }
}
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }   // no row seen: zeros
// 2^(m - top) of a state with maximum m; nothing seen: 0
__device__ __forceinline__ float state_weight(float m, float top) { return m == -INFINITY ? 0.0f : ex2(m - top); }

// The states that several CTAs left of a tile.
template <int D, typename QT>
__device__ __noinline__ void join_states(const GqaParams& p, const GqaSegment& seg, int warp, int lane) {
    const int g = lane >> 2;
    float t0 = -INFINITY, t1 = -INFINITY;
    for (int i = 0; i < seg.count; ++i) {
        const int sl = Walk::slot(seg.first + i, seg.first);
        t0 = fmaxf(t0, __ldcg(&p.ws_ml[sl * kM + g]).x);
        t1 = fmaxf(t1, __ldcg(&p.ws_ml[sl * kM + g + 8]).x);
    }
    for (int wd = warp; wd < D / 32; wd += kWarps) {
        float4 o[4] = {};
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll 4
        for (int i = 0; i < seg.count; ++i) {
            const int sl = Walk::slot(seg.first + i, seg.first);
            const float2 a = __ldcg(&p.ws_ml[sl * kM + g]), b = __ldcg(&p.ws_ml[sl * kM + g + 8]);
            const float x = state_weight(a.x, t0), y = state_weight(b.x, t1);
            s0 += a.y * x;
            s1 += b.y * y;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 v =
                    __ldcg(reinterpret_cast<const float4*>(p.ws_o) + ((int64_t)sl * (D / 8) + 4 * wd + e) * 32 + lane);
                o[e].x += v.x * x;
                o[e].y += v.y * x;
                o[e].z += v.z * y;
                o[e].w += v.w * y;
            }
        }
        write_out<D, QT>(p, seg, lane, wd, o, inverse_sum(s0), inverse_sum(s1));
    }
}

template <int D, int QP, typename QT>
__global__ void __launch_bounds__(kNT, sm_ctas<D>()) gqa_attn_kernel(const __grid_constant__ GqaParams p) {
    extern __shared__ __align__(16) unsigned char raw[];
    Smem<D, QP>& sm = *reinterpret_cast<Smem<D, QP>*>(raw);
    launch_dependents();
    grid_dependency_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    {
        Walk walk;
        const bool any = walk.template start<kNT>(p, blockIdx.x, gridDim.x, sm.part);
        if (!any) return;
        if (tid == 0) sm.walk = walk;
    }
    const GqaSegment& seg = sm.seg;
    const int32_t in_page = (1 << p.shift) - 1;
    for (;;) {
        // one copy of the walk: its state would cost every thread 40 registers
        if (tid == 0) sm.more = sm.walk.get(p, sm.seg);
        __syncthreads();
        if (!sm.more) break;
        load_queries<D, QP, QT>(p, seg, sm);
        // rows each of this lane's two vectors sees; rows that all vectors see
        const int32_t lim0 = gqa_limit(p, seg, seg.vec0 + min(g, seg.vecs - 1));
        const int32_t lim1 = gqa_limit(p, seg, seg.vec0 + min(g + 8, seg.vecs - 1));
        const int32_t all = gqa_limit(p, seg, seg.vec0);
        const int32_t end = min(seg.limit, seg.u1 * kN);
        int32_t r = seg.u0 * kN + warp * 16;
        float acc[D / 8][4];
#pragma unroll
        for (int t = 0; t < D / 8; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][i] = 0.0f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f, f0 = 0.0f, f1 = 0.0f;
        float tl0 = 0.0f, tl1 = 0.0f;
        bool flushed = false;
        Rows<D> rows;
        int64_t at = 0;
        int32_t page = 0;
        if (r < end) {
            at = (((int64_t)gqa_page(p, seg.b, r) * p.n_kv + seg.h) << p.shift) + (r & in_page);
            load_keys<D>(rows, p.k_codes + at * D, g, c);
            load_scales<D>(rows, p.scales + at, c);
            load_values<D>(rows, p.v_codes + at * D, g, c);
            if (r + kN < end) page = gqa_page(p, seg.b, r + kN);
        }
        __syncthreads();   // queries stored
        const float qs0 = sm.qs[g], qs1 = sm.qs[g + 8];
        int steps = 0;
#pragma unroll 1
        for (; r < end; r += kN) {
            const bool more = r + kN < end;
            if (more) at = (((int64_t)page * p.n_kv + seg.h) << p.shift) + ((r + kN) & in_page);
            if (r + 2 * kN < end) page = gqa_page(p, seg.b, r + 2 * kN);
            float z[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) z[t][i] = 0.0f;
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    uint32_t b0, b1;
                    e4m3x4_to_half2x2(rows.k[t][s], b0, b1);
#pragma unroll
                    for (int q = 0; q < QP; ++q) mma16816(z[t], sm.q[q][s][lane], b0, b1);
                }
            }
            if (more) load_keys<D>(rows, p.k_codes + at * D, g, c);
            float sv[4];
            {
                const float sk[4] = {rows.s[0].x, rows.s[0].z, rows.s[1].x, rows.s[1].z};
                sv[0] = rows.s[0].y;
                sv[1] = rows.s[0].w;
                sv[2] = rows.s[1].y;
                sv[3] = rows.s[1].w;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) z[t][i] = z[t][i] * sk[2 * t + (i & 1)] * (i < 2 ? qs0 : qs1);
            }
            if (more) load_scales<D>(rows, p.scales + at, c);
            bool hide[2][4] = {};
            if (r + 16 > all) {   // some vector sees these rows in part
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    bool bad = false;
#pragma unroll
                    for (int w = 0; w < D / 32; ++w) {
                        const uint32_t x = rows.v[k][w], nan = (((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
                        bad |= nan != 0u;
                        rows.v[k][w] = x ^ nan;
                    }
                    const unsigned who = __ballot_sync(kFull, bad);
                    if (who & (0x11111111u << c)) sv[k] = __uint_as_float(0x7fffffffu);
                }
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        hide[t][i] = r + 8 * t + 2 * c + (i & 1) >= (i < 2 ? lim0 : lim1);
                        if (hide[t][i]) z[t][i] = -INFINITY;
                    }
            }
            float pr[2][4], w[2][4];
            bool lift = false;
            {
                const float a0 = m0 == -INFINITY ? 0.0f : m0, a1 = m1 == -INFINITY ? 0.0f : m1;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        lift |= z[t][i] > (i < 2 ? m0 : m1) + 8.0f;
                        pr[t][i] = ex2(z[t][i] - (i < 2 ? a0 : a1));
                        w[t][i] = hide[t][i] ? 0.0f : pr[t][i] * (sv[2 * t + (i & 1)] * (i < 2 ? f0 : f1));
                        lift |= fabsf(w[t][i]) > 60000.0f;
                    }
            }
            if (__any_sync(kFull, lift)) {
                // new maxima, new factors f, and what is summed so far brought to them
                float n0 = m0, n1 = m1;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    n0 = fmaxf(n0, fmaxf(z[t][0], z[t][1]));
                    n1 = fmaxf(n1, fmaxf(z[t][2], z[t][3]));
                }
#pragma unroll
                for (int o = 1; o <= 2; o <<= 1) {
                    n0 = fmaxf(n0, __shfl_xor_sync(kFull, n0, o));
                    n1 = fmaxf(n1, __shfl_xor_sync(kFull, n1, o));
                }
                const float a0 = n0 == -INFINITY ? 0.0f : n0, a1 = n1 == -INFINITY ? 0.0f : n1;
                float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        pr[t][i] = ex2(z[t][i] - (i < 2 ? a0 : a1));
                        w[t][i] = hide[t][i] ? 0.0f : pr[t][i] * sv[2 * t + (i & 1)];
                        if (i < 2) t0 = fmaxf(t0, fabsf(w[t][i]));
                        else t1 = fmaxf(t1, fabsf(w[t][i]));
                    }
#pragma unroll
                for (int o = 1; o <= 2; o <<= 1) {
                    t0 = fmaxf(t0, __shfl_xor_sync(kFull, t0, o));
                    t1 = fmaxf(t1, __shfl_xor_sync(kFull, t1, o));
                }
                const float d0 = state_weight(m0, a0), d1 = state_weight(m1, a1);
                // the largest weight so far, at most 2^14 / f, against the step's
                const float b0 = fmaxf(t0, f0 > 0.0f ? d0 * 0x1p14f / f0 : 0.0f);
                const float b1 = fmaxf(t1, f1 > 0.0f ? d1 * 0x1p14f / f1 : 0.0f);
                const float h0 = b0 > 0.0f ? fminf(0x1p14f / b0, 0x1p100f) : f0;
                const float h1 = b1 > 0.0f ? fminf(0x1p14f / b1, 0x1p100f) : f1;
                const float k0 = f0 > 0.0f ? d0 * (h0 / f0) : 0.0f, k1 = f1 > 0.0f ? d1 * (h1 / f1) : 0.0f;
#pragma unroll
                for (int t = 0; t < D / 8; ++t) {
                    acc[t][0] *= k0;
                    acc[t][1] *= k0;
                    acc[t][2] *= k1;
                    acc[t][3] *= k1;
                }
                if (flushed) {
#pragma unroll 4
                    for (int t = 0; t < D / 8; ++t) {
                        float4 v = sm.tot[warp][t][lane];
                        v.x *= k0;
                        v.y *= k0;
                        v.z *= k1;
                        v.w *= k1;
                        sm.tot[warp][t][lane] = v;
                    }
                }
                l0 *= d0;
                l1 *= d1;
                tl0 *= d0;
                tl1 *= d1;
                m0 = n0;
                m1 = n1;
                f0 = h0;
                f1 = h1;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[t][i] *= i < 2 ? f0 : f1;
            }
            l0 += (pr[0][0] + pr[0][1]) + (pr[1][0] + pr[1][1]);
            l1 += (pr[0][2] + pr[0][3]) + (pr[1][2] + pr[1][3]);
            uint4 hi, lo;
            hi.x = pack_half2(w[0][0], w[0][1]);
            hi.y = pack_half2(w[0][2], w[0][3]);
            hi.z = pack_half2(w[1][0], w[1][1]);
            hi.w = pack_half2(w[1][2], w[1][3]);
            {
                const float2 x = unpack_half2(hi.x), y = unpack_half2(hi.y), u = unpack_half2(hi.z), v = unpack_half2(hi.w);
                lo.x = pack_half2(w[0][0] - x.x, w[0][1] - x.y);
                lo.y = pack_half2(w[0][2] - y.x, w[0][3] - y.y);
                lo.z = pack_half2(w[1][0] - u.x, w[1][1] - u.y);
                lo.w = pack_half2(w[1][2] - v.x, w[1][3] - v.y);
            }
#pragma unroll
            for (int wd = 0; wd < D / 32; ++wd) {
                uint32_t a[4], b[4];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t x = rows.v[2 * k][wd], y = rows.v[2 * k + 1][wd];
                    uint32_t* dst = k == 0 ? a : b;
                    e4m3x4_to_half2x2(__byte_perm(x, y, 0x5140), dst[0], dst[1]);
                    e4m3x4_to_half2x2(__byte_perm(x, y, 0x7362), dst[2], dst[3]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    mma16816(acc[4 * wd + e], hi, a[e], b[e]);
                    mma16816(acc[4 * wd + e], lo, a[e], b[e]);
                }
            }
            if (more) load_values<D>(rows, p.v_codes + at * D, g, c);
            if (++steps == kFlush) {
                steps = 0;
#pragma unroll
                for (int t = 0; t < D / 8; ++t) {
                    float4 v = flushed ? sm.tot[warp][t][lane] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    v.x += acc[t][0];
                    v.y += acc[t][1];
                    v.z += acc[t][2];
                    v.w += acc[t][3];
                    sm.tot[warp][t][lane] = v;
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[t][i] = 0.0f;
                }
                flushed = true;
                tl0 += l0;
                tl1 += l1;
                l0 = 0.0f;
                l1 = 0.0f;
            }
        }
        // the warp's state to shared memory
#pragma unroll
        for (int t = 0; t < D / 8; ++t) {
            float4 v = flushed ? sm.tot[warp][t][lane] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            v.x += acc[t][0];
            v.y += acc[t][1];
            v.z += acc[t][2];
            v.w += acc[t][3];
            sm.tot[warp][t][lane] = v;
        }
        tl0 += l0;
        tl1 += l1;
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
            tl0 += __shfl_xor_sync(kFull, tl0, o);
            tl1 += __shfl_xor_sync(kFull, tl1, o);
        }
        if (c == 0) {
            sm.m[warp][g] = m0;
            sm.m[warp][g + 8] = m1;
            sm.l[warp][g] = tl0;
            sm.l[warp][g + 8] = tl1;
            sm.f[warp][g] = f0;
            sm.f[warp][g + 8] = f1;
        }
        __syncthreads();
        // the warps' states joined, for the two vectors of this lane
        float top0 = -INFINITY, top1 = -INFINITY, sum0 = 0.0f, sum1 = 0.0f, k0[kWarps], k1[kWarps];
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            top0 = fmaxf(top0, sm.m[i][g]);
            top1 = fmaxf(top1, sm.m[i][g + 8]);
        }
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            const float x = state_weight(sm.m[i][g], top0), y = state_weight(sm.m[i][g + 8], top1);
            sum0 += sm.l[i][g] * x;
            sum1 += sm.l[i][g + 8] * y;
            k0[i] = sm.f[i][g] > 0.0f ? x / sm.f[i][g] : 0.0f;
            k1[i] = sm.f[i][g + 8] > 0.0f ? y / sm.f[i][g + 8] : 0.0f;
        }
        const bool whole = seg.slot < 0;
        if (!whole && warp == 0 && c == 0) {
            p.ws_ml[seg.slot * kM + g] = make_float2(top0, sum0);
            p.ws_ml[seg.slot * kM + g + 8] = make_float2(top1, sum1);
        }
        for (int wd = warp; wd < D / 32; wd += kWarps) {
            float4 o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                o[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < kWarps; ++i) {
                    const float4 v = sm.tot[i][4 * wd + e][lane];
                    o[e].x += v.x * k0[i];
                    o[e].y += v.y * k0[i];
                    o[e].z += v.z * k1[i];
                    o[e].w += v.w * k1[i];
                }
                if (!whole) reinterpret_cast<float4*>(p.ws_o)[((int64_t)seg.slot * (D / 8) + 4 * wd + e) * 32 + lane] = o[e];
            }
            if (whole) write_out<D, QT>(p, seg, lane, wd, o, inverse_sum(sum0), inverse_sum(sum1));
        }
        if (!whole) {
            // the CTA that comes last joins the tile's states, in the rows' order
            __threadfence();
            __syncthreads();
            if (tid == 0) sm.last = atomicAdd(p.tickets + seg.first, 1u) == (uint32_t)(seg.count - 1);
            __syncthreads();
            if (sm.last) {
                __threadfence();
                if (tid == 0) p.tickets[seg.first] = 0u;
                join_states<D, QT>(p, seg, warp, lane);
            }
        }
        if (warp == 0) {
            Walk walk = sm.walk;
            walk.next(p);
            __syncwarp();
            if (lane == 0) sm.walk = walk;
        }
        __syncthreads();   // the totals and queries are free for the next tile
    }
}

template <int D, int QP, typename QT>
cudaError_t launch_dims(const GqaParams& p, cudaStream_t stream) {
    constexpr size_t smem = sizeof(Smem<D, QP>);
    const cudaError_t e =
        cudaFuncSetAttribute(gqa_attn_kernel<D, QP, QT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_chained(gqa_attn_kernel<D, QP, QT>, 152 * sm_ctas<D>(), kNT, smem, stream, p);
}
template <int D>
cudaError_t launch_type(const GqaParams& p, kvq_dtype dt, cudaStream_t stream) {
    return dt == KVQ_BF16 ? launch_dims<D, 1, __nv_bfloat16>(p, stream) : launch_dims<D, 2, float>(p, stream);
}

constexpr size_t kTicketBytes = 4096;
static_assert(kGqaMaxCtas * 4 <= kTicketBytes, "a ticket a CTA");

}  // namespace

// Error word and tickets, the cut tiles' maxima and sums, their contexts.
size_t gqa_attn_workspace_bytes(int32_t head_dim) {
    return kWsHeader + kTicketBytes + (size_t)2 * kGqaMaxCtas * kM * (sizeof(float2) + head_dim * sizeof(float));
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
    p.tickets = reinterpret_cast<uint32_t*>(ws + kWsHeader);
    p.ws_ml = reinterpret_cast<float2*>(ws + kWsHeader + kTicketBytes);
    p.ws_o = reinterpret_cast<float*>(p.ws_ml + 2 * kGqaMaxCtas * kM);
    timing_mark(stream, 0);
    cudaError_t e;
    switch (c.head_dim) {
        case 64: e = launch_type<64>(p, c.dtype, stream); break;
        case 128: e = launch_type<128>(p, c.dtype, stream); break;
        case 256: e = launch_type<256>(p, c.dtype, stream); break;
        default: return cudaErrorInvalidValue;
    }
    timing_mark(stream, 1);
    timing_mark(stream, 2);
    return e;
}

}  // namespace kvq
