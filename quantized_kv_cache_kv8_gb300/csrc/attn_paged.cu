// attn_paged.cu -- attention of new tokens over paged quantized rows: the exact
// (fp32) kernel, the merge of cut tiles, and the launch.
//
// The exact kernel: a CTA walks over (query tile, run of row steps) segments
// (paged_common.cuh) with 32 query vectors and 32 rows a step in shared memory,
// both in f32; the rows are the codes' values, the row scales stay outside both
// sums as in the contiguous kernels.  Scores: a thread takes 2 vectors x 2
// rows, so four 16-byte reads serve 16 multiply-adds (a head and a row a thread
// needs two for 4).  Context: a thread takes 8 vectors x 8 dims in registers.
// Sums run in three levels -- the 32 rows of a step, 32 steps, and the totals of those in
// the workspace, two f32 each -- so that roundings that all point one way stay under
// (32 + 32) 2^-24 whatever the length (with first sums of 1,024 rows, 131,072 rows alike
// behind one that outweighs them came out 4.6e-5 off).  What bounds it is latency: one CTA of 8 warps an SM, and loads,
// scores and context of a step one after the other, 11 TFLOP/s for 16 sequences of 60 to
// 1000 rows x 32 heads (44 us), a seventh of the FMA rate; 29 us for 4 sequences of 100 to
// 700 rows x 16 heads.
#include "paged_common.cuh"

#include <math.h>
#include <type_traits>

namespace kvq {
namespace {

constexpr int kNT = 256;
constexpr int kM = PagedSimt::kM, kN = PagedSimt::kN;
constexpr int kXS = 580;             // row stride in floats (4 banks apart)
constexpr int kPS = kM + 4;          // weights: [row][vector]
constexpr int kFlush = 1024 / kN;    // steps per block sum
constexpr size_t kSmemFloats = (size_t)(kM + kN) * kXS + kN * 2 + (size_t)kN * kPS + 3 * kM + 16;
constexpr size_t kSmem = kSmemFloats * 4 + kN * 4 + kM * 8 + kWalkScratch<kNT> * 8 + 16;

__device__ __forceinline__ void store_out(float* o, int64_t i, float4 v) { *reinterpret_cast<float4*>(o + i) = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16* o, int64_t i, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    uint2 w;
    w.x = *reinterpret_cast<const uint32_t*>(&a);
    w.y = *reinterpret_cast<const uint32_t*>(&b);
    *reinterpret_cast<uint2*>(o + i) = w;
}
__device__ __forceinline__ void store_out1(float* o, int64_t i, float v) { o[i] = v; }
__device__ __forceinline__ void store_out1(__nv_bfloat16* o, int64_t i, float v) { o[i] = __float2bfloat16_rn(v); }

// The context of one query vector, normalized and in the rotated domain, held
// by a warp (lane + 32 k): unrotated and written.
template <typename OT>
__device__ __forceinline__ void unrotate_out(const PagedParams& p, float (&v)[16], OT* out, int64_t at, int lane) {
    warp_fwht<512>(v, lane);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int i = lane + 32 * k;
        const float y = __fmul_rn(v[k], p.kn[0]);
        store_out1(out, at + i, sign_neg(p.signs, 0, i) ? -y : y);
    }
}

template <bool TQ4, bool BF16>
__global__ void __launch_bounds__(kNT, 1) paged_exact_kernel(const __grid_constant__ PagedParams p) {
    using OT = typename std::conditional<BF16, __nv_bfloat16, float>::type;
    launch_dependents();
    extern __shared__ float4 smem4[];
    float* qs = reinterpret_cast<float*>(smem4);
    float* xs = qs + kM * kXS;
    float* sc = xs + kN * kXS;
    float* P = sc + kN * 2;
    float* alpha = P + kN * kPS;
    float* scale = alpha + kM;   // what a vector's total counts by now
    float* lost_l = scale + kM;  // what additions of the row sum rounded away
    float* lvs = lost_l + kM;
    int32_t* prow = reinterpret_cast<int32_t*>(lvs + 16);
    int64_t* lim = reinterpret_cast<int64_t*>(prow + kN);
    int64_t* part = lim + kM;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t cta = blockIdx.x;
    if (tid < 16) lvs[tid] = p.lv[tid];
    grid_dependency_wait();
    if (tid < 4) p.ws_desc[cta * 4 + tid] = 0;
    PagedWalk<PagedSimt> walk;
    if (!walk.template start<kNT>(p, cta, gridDim.x, part)) return;

    const int ty = tid >> 4, tx = tid & 15;   // scores: vectors 2 ty, 2 ty + 1; rows tx, tx + 16
    const int cq = tid >> 6, cc = tid & 63;   // context: vectors 8 cq ..; dims 4 cc .., 256 + 4 cc ..
    Segment g;
    for (; walk.get(p, g); walk.next(p)) {
        __syncthreads();
        for (int i = tid; i < kM * kMlaD; i += kNT) {
            const int r = i / kMlaD, d = i - r * kMlaD;
            qs[r * kXS + d] = r < g.rows ? load_q<BF16>(p.q, (g.row0 + r) * kMlaD + d) : 0.0f;
        }
        if (tid < kM) {
            lim[tid] = tid < g.rows ? row_limit(p, g, tid) : 0;
            scale[tid] = 1.0f;
            lost_l[tid] = 0.0f;
        }
        __syncthreads();
        if (TQ4) {
            for (int r = warp; r < kM; r += kNT / 32) {
                float* qr = qs + r * kXS;
                float v[16], w[2];
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = sign_neg(p.signs, 0, lane + 32 * k) ? -qr[lane + 32 * k] : qr[lane + 32 * k];
                warp_fwht<512>(v, lane);
#pragma unroll
                for (int k = 0; k < 16; ++k) qr[lane + 32 * k] = __fmul_rn(v[k], p.kn[0]);
                qr += kMlaDL;
#pragma unroll
                for (int k = 0; k < 2; ++k) w[k] = sign_neg(p.signs, 1, lane + 32 * k) ? -qr[lane + 32 * k] : qr[lane + 32 * k];
                warp_fwht<64>(w, lane);
#pragma unroll
                for (int k = 0; k < 2; ++k) qr[lane + 32 * k] = __fmul_rn(w[k], p.kn[1]);
            }
            __syncthreads();
        }
        float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f}, l_blk[2] = {0.f, 0.f};
        float o[8][8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) o[i][k] = 0.0f;
        // totals of the block sums, in the walker's second slot (free until its last segment
        // ends), and what their additions rounded away
        float* total = p.ws_o + ((2 * cta + 1) * kM + 8 * cq) * kMlaDV + 4 * cc;
        float* lost = p.ws_c + (cta * kM + 8 * cq) * kMlaDV + 4 * cc;
        bool folded = false;
        // 4 dims d .. of vector i: o into their total (exactly, with `lost`), or the total into o
        auto fold4 = [&](int i, int d, float* o4, bool back) {
            float4* to = reinterpret_cast<float4*>(total + i * kMlaDV + d);
            float4* lo = reinterpret_cast<float4*>(lost + i * kMlaDV + d);
            const float f = scale[8 * cq + i];
            float t[4] = {}, c[4] = {};
            if (folded) {
                const float4 a = *to, b = *lo;
                const float va[4] = {a.x, a.y, a.z, a.w}, vb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    t[k] = __fmul_rn(va[k], f);
                    c[k] = __fmul_rn(vb[k], f);
                }
            }
            if (back) {
#pragma unroll
                for (int k = 0; k < 4; ++k) o4[k] = __fadd_rn(__fadd_rn(o4[k], c[k]), t[k]);
                return;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float s = __fadd_rn(t[k], o4[k]), part = __fsub_rn(s, t[k]);
                c[k] = __fadd_rn(c[k], __fadd_rn(__fsub_rn(t[k], __fsub_rn(s, part)), __fsub_rn(o4[k], part)));
                t[k] = s;
                o4[k] = 0.0f;
            }
            *to = make_float4(t[0], t[1], t[2], t[3]);
            *lo = make_float4(c[0], c[1], c[2], c[3]);
        };
        const int64_t end = row_limit(p, g, g.rows - 1);   // rows any vector of the tile sees
        int steps = 0;
        for (int64_t u = g.u0; u < g.u1; ++u) {
            const int64_t t0 = u * kN;
            const int nt = (int)max((int64_t)0, min((int64_t)kN, end - t0));
            if (tid < kN) prow[tid] = tid < nt ? paged_row(p, g.b, t0 + tid) : 0;
            __syncthreads();
            constexpr int kWords = TQ4 ? kMlaD / 8 : kMlaD / 4;   // 32-bit code words of a row
            for (int w = tid; w < kN * kWords; w += kNT) {
                const int r = w / kWords, c = w - r * kWords;
                uint32_t x = 0u;
                if (r < nt) x = __ldg(reinterpret_cast<const uint32_t*>(p.codes + (int64_t)prow[r] * (kWords * 4)) + c);
                if (TQ4) {
                    float f[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) f[k] = r < nt ? lvs[(x >> (4 * k)) & 15u] : 0.0f;
                    *reinterpret_cast<float4*>(xs + r * kXS + 8 * c) = make_float4(f[0], f[1], f[2], f[3]);
                    *reinterpret_cast<float4*>(xs + r * kXS + 8 * c + 4) = make_float4(f[4], f[5], f[6], f[7]);
                } else {
                    *reinterpret_cast<float4*>(xs + r * kXS + 4 * c) = e4m3x4_to_float4(x);
                }
            }
            if (tid < kN) {
                const float* s = p.scales + (int64_t)prow[tid] * p.n_blocks;
                const float2 v = tid < nt ? row_scales(s[0], s[p.n_blocks - 1]) : make_float2(0.0f, 0.0f);
                sc[2 * tid] = v.x;
                sc[2 * tid + 1] = v.y;
            }
            __syncthreads();
            {
                // dot products over runs of 128 dims in four interleaved sums,
                // then over the runs: 32 terms a chain keep the f32 rounding of
                // a score near 2^-24 sqrt(32) of its largest run
                float dot[2][2] = {}, rope[2][2] = {};
                const float *q0 = qs + 2 * ty * kXS, *q1 = q0 + kXS, *x0 = xs + tx * kXS, *x1 = xs + (tx + 16) * kXS;
                auto run = [&](int d0, int d1, float (&sum)[2][2]) {
                    float4 c[2][2] = {};
#pragma unroll 8
                    for (int d = d0; d < d1; d += 4) {
                        const float4 qv[2] = {*reinterpret_cast<const float4*>(q0 + d), *reinterpret_cast<const float4*>(q1 + d)};
                        const float4 xv[2] = {*reinterpret_cast<const float4*>(x0 + d), *reinterpret_cast<const float4*>(x1 + d)};
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                c[i][k].x = fmaf(qv[i].x, xv[k].x, c[i][k].x);
                                c[i][k].y = fmaf(qv[i].y, xv[k].y, c[i][k].y);
                                c[i][k].z = fmaf(qv[i].z, xv[k].z, c[i][k].z);
                                c[i][k].w = fmaf(qv[i].w, xv[k].w, c[i][k].w);
                            }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            sum[i][k] += (c[i][k].x + c[i][k].y) + (c[i][k].z + c[i][k].w);
                };
#pragma unroll 1
                for (int d = 0; d < kMlaDL; d += 128) run(d, d + 128, dot);
                run(kMlaDL, kMlaD, rope);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int64_t seen = lim[2 * ty + i];
                    float z[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int r = tx + 16 * k;
                        const float s = p.sm_scale * (sc[2 * r] * dot[i][k] + sc[2 * r + 1] * rope[i][k]);
                        z[k] = t0 + r < seen ? s : -INFINITY;
                    }
                    float top = fmaxf(z[0], z[1]);
#pragma unroll
                    for (int off = 8; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
                    const float m_new = fmaxf(m_run[i], top);
                    const float m_ref = m_new == -INFINITY ? 0.0f : m_new;   // nothing seen yet: weights 0
                    const float a = m_run[i] == -INFINITY ? 0.0f : expf(m_run[i] - m_ref);
                    float sum = 0.0f;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int r = tx + 16 * k;
                        const float w = expf(z[k] - m_ref);
                        sum += w;
                        P[r * kPS + 2 * ty + i] = z[k] == -INFINITY ? 0.0f : w * sc[2 * r];
                    }
#pragma unroll
                    for (int off = 8; off >= 1; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
                    l_blk[i] = l_blk[i] * a + sum;
                    l_run[i] *= a;
                    m_run[i] = m_new;
                    if (tx == 0) {
                        alpha[2 * ty + i] = a;
                        scale[2 * ty + i] *= a;
                    }
                }
            }
            __syncthreads();
            {
                float step[8][8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int k = 0; k < 8; ++k) step[i][k] = 0.0f;
                for (int t = 0; t < nt; ++t) {
                    const float4 xa = *reinterpret_cast<const float4*>(xs + t * kXS + 4 * cc);
                    const float4 xb = *reinterpret_cast<const float4*>(xs + t * kXS + 256 + 4 * cc);
                    const float4 pa = *reinterpret_cast<const float4*>(P + t * kPS + 8 * cq);
                    const float4 pb = *reinterpret_cast<const float4*>(P + t * kPS + 8 * cq + 4);
                    const float w[8] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
                    float x[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
                    // a NaN code (finite here) reaches the vectors that see its row by their weights
                    if (!TQ4)
#pragma unroll
                        for (int k = 0; k < 8; ++k) x[k] = fmaxf(x[k], -448.0f);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int k = 0; k < 8; ++k) step[i][k] = fmaf(w[i], x[k], step[i][k]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float al = alpha[8 * cq + i];
#pragma unroll
                    for (int k = 0; k < 8; ++k) o[i][k] = fmaf(o[i][k], al, step[i][k]);
                }
            }
            if (++steps == kFlush) {
                steps = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    fold4(i, 0, o[i], false);
                    fold4(i, 256, o[i] + 4, false);
                }
                folded = true;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = 2 * ty + i;
                    const float s = __fadd_rn(l_run[i], l_blk[i]), part = __fsub_rn(s, l_run[i]);
                    const float c = __fmul_rn(lost_l[r], scale[r]) +
                                    __fadd_rn(__fsub_rn(l_run[i], __fsub_rn(s, part)), __fsub_rn(l_blk[i], part));
                    __syncwarp();
                    if (tx == 0) lost_l[r] = c;
                    l_run[i] = s;
                    l_blk[i] = 0.0f;
                }
                __syncthreads();   // every thread has read its scales
                if (tid < kM) scale[tid] = 1.0f;
            }
            __syncthreads();
        }
        int64_t parts;
        const int64_t slot = walk.slot(g, cta, &parts);
#pragma unroll
        for (int i = 0; i < 2; ++i) l_run[i] += l_blk[i] + lost_l[2 * ty + i] * scale[2 * ty + i];
        if (folded)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                fold4(i, 0, o[i], true);
                fold4(i, 256, o[i] + 4, true);
            }
        if (slot >= 0) {
            if (tx == 0)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float* ml = p.ws_ml + (slot * kM + 2 * ty + i) * 2;
                    ml[0] = m_run[i];
                    ml[1] = l_run[i];
                }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float* dst = p.ws_o + (slot * kM + 8 * cq + i) * kMlaDV;
                *reinterpret_cast<float4*>(dst + 4 * cc) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
                *reinterpret_cast<float4*>(dst + 256 + 4 * cc) = make_float4(o[i][4], o[i][5], o[i][6], o[i][7]);
            }
            if (parts > 0 && tid == 0) {
                p.ws_desc[cta * 4] = parts;
                p.ws_desc[cta * 4 + 1] = g.row0;
                p.ws_desc[cta * 4 + 2] = g.rows;
            }
            continue;
        }
        if (tx == 0)
#pragma unroll
            for (int i = 0; i < 2; ++i) alpha[2 * ty + i] = l_run[i] == 0.0f ? 0.0f : 1.0f / l_run[i];
        __syncthreads();
        OT* out = static_cast<OT*>(p.out);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 8 * cq + i;
            const float f = alpha[r];
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = o[i][k] * f;
            const float4 a = make_float4(v[0], v[1], v[2], v[3]), b = make_float4(v[4], v[5], v[6], v[7]);
            if (TQ4) {
                *reinterpret_cast<float4*>(qs + r * kXS + 4 * cc) = a;
                *reinterpret_cast<float4*>(qs + r * kXS + 256 + 4 * cc) = b;
            } else if (r < g.rows) {
                store_out(out, (g.row0 + r) * kMlaDV + 4 * cc, a);
                store_out(out, (g.row0 + r) * kMlaDV + 256 + 4 * cc, b);
            }
        }
        if (TQ4) {
            __syncthreads();
            for (int r = warp; r < g.rows; r += kNT / 32) {
                float v[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = qs[r * kXS + lane + 32 * k];
                unrotate_out(p, v, out, (g.row0 + r) * kMlaDV, lane);
            }
        }
    }
}

constexpr int kMergeRows = 4, kMergeNT = 128 * kMergeRows, kMergeCtas = 304;

// Joins the parts of cut tiles by log-sum-exp: 4 vectors at a time, 128 threads
// with 4 dims each to a vector.  Each CTA lists the walkers that began a cut tile
// and takes its share of their vectors (a CTA for every walker and group of vectors
// would be 2,400, most of them with nothing to do).
template <bool TQ4, bool BF16, int M>
__global__ void __launch_bounds__(kMergeNT) paged_merge_kernel(const __grid_constant__ PagedParams p) {
    using OT = typename std::conditional<BF16, __nv_bfloat16, float>::type;
    constexpr int kWalkers = M == PagedTensor::kM ? kPagedPairs : kPagedCtas;
    static_assert(kWalkers <= kMergeNT, "a thread a walker");
    __shared__ float ov[kMergeRows][kMlaDV];
    constexpr int kListWarps = (kWalkers + 31) / 32;
    __shared__ int32_t cut[kWalkers], in_warp[kListWarps];
    const int sub = threadIdx.x >> 7, tid = threadIdx.x & 127, lane = tid & 31, warp = threadIdx.x >> 5;
    launch_dependents();
    grid_dependency_wait();
    // the walkers with a cut tile, in order: every CTA has the same list
    const bool mine = threadIdx.x < kWalkers && p.ws_desc[threadIdx.x * 4] > 0;
    const unsigned mask = __ballot_sync(kFull, mine);
    if (lane == 0 && warp < kListWarps) in_warp[warp] = __popc(mask);
    __syncthreads();
    int before = 0, n_cut = 0;
#pragma unroll
    for (int w = 0; w < kListWarps; ++w) {
        before += w < warp ? in_warp[w] : 0;
        n_cut += in_warp[w];
    }
    if (mine) cut[before + __popc(mask & ((1u << lane) - 1u))] = threadIdx.x;
    __syncthreads();
    constexpr int kGroups = M / kMergeRows;
    for (int item = blockIdx.x; item < n_cut * kGroups; item += gridDim.x) {
        const int64_t cta = cut[item / kGroups];
        const int r = kMergeRows * (item % kGroups) + sub;
        const int64_t parts = p.ws_desc[cta * 4], row0 = p.ws_desc[cta * 4 + 1];
        const bool live = r < p.ws_desc[cta * 4 + 2];
        float Mx = -INFINITY, L = 0.0f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kBatch = 8;
        for (int64_t c0 = 0; live && c0 < parts; c0 += kBatch) {
            float mv[kBatch], lw[kBatch];
            float4 v[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                mv[k] = -INFINITY;
                lw[k] = 0.0f;
                v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c0 + k < parts) {
                    // the beginning lies in this CTA's second slot, the rest in the first slots of the CTAs after it
                    const int64_t row = (c0 + k == 0 ? 2 * cta + 1 : 2 * (cta + c0 + k)) * M + r;
                    const float2 ml = *reinterpret_cast<const float2*>(p.ws_ml + row * 2);
                    mv[k] = ml.x;
                    lw[k] = ml.y;
                    v[k] = *reinterpret_cast<const float4*>(p.ws_o + row * kMlaDV + 4 * tid);
                }
            }
            float mb = Mx;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) mb = fmaxf(mb, mv[k]);
            const float ref = mb == -INFINITY ? 0.0f : mb;   // parts without a visible row weigh 0
            const float keep = expf(Mx - ref);
            L *= keep;
            acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const float w = expf(mv[k] - ref);
                L = fmaf(w, lw[k], L);
                acc.x = fmaf(w, v[k].x, acc.x);
                acc.y = fmaf(w, v[k].y, acc.y);
                acc.z = fmaf(w, v[k].z, acc.z);
                acc.w = fmaf(w, v[k].w, acc.w);
            }
            Mx = mb;
        }
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;   // no visible row: zeros
        acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        OT* out = static_cast<OT*>(p.out);
        const int64_t at = (row0 + r) * kMlaDV;
        if (!TQ4) {
            if (live) store_out(out, at + 4 * tid, acc);
            continue;
        }
        *reinterpret_cast<float4*>(ov[sub] + 4 * tid) = acc;
        __syncthreads();
        if (live && tid < 32) {
            float v[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = ov[sub][lane + 32 * k];
            unrotate_out(p, v, out, at, lane);
        }
        __syncthreads();   // ov is read before the next item's values
    }
}

template <bool TQ4, bool BF16>
cudaError_t launch_exact(const PagedParams& p, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(paged_exact_kernel<TQ4, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmem);
    if (e != cudaSuccess) return e;
    return launch_chained(paged_exact_kernel<TQ4, BF16>, kPagedCtas, kNT, kSmem, stream, p);
}

template <bool TQ4, bool BF16, int M>
cudaError_t launch_merge(const PagedParams& p, cudaStream_t stream) {
    return launch_chained(paged_merge_kernel<TQ4, BF16, M>, kMergeCtas, kMergeNT, 0, stream, p);
}

// query vectors of partial state: two tiles a walker
constexpr int64_t state_rows(bool tensor) {
    return tensor ? 2 * kPagedPairs * PagedTensor::kM : 2 * kPagedCtas * PagedSimt::kM;
}

}  // namespace

size_t paged_workspace_bytes(bool tensor) {
    return kWsHeader + (size_t)kPagedCtas * 4 * sizeof(int64_t) + (size_t)state_rows(tensor) * (kMlaDV + 2) * sizeof(float) +
           (tensor ? (size_t)kPagedCtas * 256 * sizeof(float2) : (size_t)kPagedCtas * kM * kMlaDV * sizeof(float));
}

cudaError_t launch_attn_paged(kvq_format fmt, const kvq_mla_layout& L, bool tensor, const void* q, kvq_dtype dt,
                              int64_t n_tok, int32_t n_heads, int32_t n_seq, const int64_t* cu_q, const uint8_t* codes,
                              const float* scales, const int32_t* table, int32_t table_stride,
                              const int64_t* kv_lens, int32_t page_rows, int32_t n_pages, float sm_scale, void* out,
                              void* workspace, cudaStream_t stream) {
    PagedParams p{};
    p.n_seq = n_seq;
    p.n_heads = n_heads;
    p.h_inv = ~0ull / (uint64_t)n_heads;
    p.q = q;
    p.out = out;
    p.codes = codes;
    p.scales = scales;
    p.cu_q = cu_q;
    p.kv_lens = kv_lens;
    p.table = table;
    p.table_stride = table_stride;
    while ((1 << p.shift) < page_rows) ++p.shift;
    p.n_pages = n_pages;
    p.n_blocks = L.n_blocks;
    p.max_tok = n_tok;
    p.sm_scale = sm_scale;
    char* ws = static_cast<char*>(workspace);
    p.err = reinterpret_cast<int32_t*>(ws);
    p.exact_count = reinterpret_cast<uint32_t*>(ws + 16);
    p.stall_polls = test_stall_polls();
    p.wait_limit = p.stall_polls > 0 ? p.stall_polls : kWaitLimit;
    p.ws_desc = reinterpret_cast<int64_t*>(ws + kWsHeader);
    p.ws_o = reinterpret_cast<float*>(ws + kWsHeader + (size_t)kPagedCtas * 4 * sizeof(int64_t));
    p.ws_ml = p.ws_o + state_rows(tensor) * kMlaDV;
    p.ws_c = p.ws_ml + state_rows(tensor) * 2;
    p.ws_l = reinterpret_cast<float2*>(p.ws_c);
    if (fmt == KVQ_TQ4) {
        p.signs = tq4_sign_words(L);
        p.kn[0] = (float)(1.0 / sqrt((double)L.block_dim[0]));
        p.kn[1] = (float)(1.0 / sqrt((double)L.block_dim[1]));
        const Codebook16 cb = tq4_codebook();
        for (int k = 0; k < 16; ++k) p.lv[k] = cb.lv[k];
    }
    const bool tq4 = fmt == KVQ_TQ4, bf16 = dt == KVQ_BF16;
    timing_mark(stream, 0);
    cudaError_t e;
    if (tensor) e = launch_paged_tensor(fmt, p, stream);
    else if (tq4) e = bf16 ? launch_exact<true, true>(p, stream) : launch_exact<true, false>(p, stream);
    else e = bf16 ? launch_exact<false, true>(p, stream) : launch_exact<false, false>(p, stream);
    if (e != cudaSuccess) return e;
    timing_mark(stream, 1);
    if (tensor) e = tq4 ? launch_merge<true, true, PagedTensor::kM>(p, stream) : launch_merge<false, true, PagedTensor::kM>(p, stream);
    else if (tq4) e = bf16 ? launch_merge<true, true, PagedSimt::kM>(p, stream) : launch_merge<true, false, PagedSimt::kM>(p, stream);
    else e = bf16 ? launch_merge<false, true, PagedSimt::kM>(p, stream) : launch_merge<false, false, PagedSimt::kM>(p, stream);
    timing_mark(stream, 2);
    return e;
}

}  // namespace kvq
