// rope.cu -- rotary positions with one or several axes, fused with the paged
// append: the step's queries are rotated into place and its new rows rotated,
// quantized and stored in their slots, in one launch.
//
// Pair i of the rotary dims turns by the angle pos[axis_i] * w_i, w_i the pair's
// inverse frequency: (u, v) -> (u cos - v sin, v cos + u sin).  An angle in f32
// is wrong by 2^-24 of its own size (0.06 rad at position 10^6), so the phase
// is kept in turns as a 64-bit fraction: inc_i = w_i / 2 pi * 2^64 on the host,
// whole turns dropped, pos * inc_i mod 2^64 on the device, exact but for the rounding of
// inc_i (2^-53 of w_i, and down to a multiple of 2^-64 turns); its signed value over 2^63 goes to sincospi in f32.
//
// What bounds it: memory, 128 bytes of query in and out per head (2048 tokens
// x 128 heads: 67 MB, 10 us at 6.8 TB/s; measured 14.3 us, 5.0 TB/s, and what keeps it
// from the rest is not known); a decode step only its latency (8 tokens 4.9 us).  The
// cos and sin of a token are shared by its heads, so a CTA tabulates them in
// shared memory for the tokens it serves and then runs through its share of
// the (token, head, 16 bytes) units.  Rows take a warp each, in CTAs of their
// own that come first: a row's chain (load, rotate, amax or rotation, codes) is
// the longest of the launch.
#include "encode_common.cuh"
#include "paged.cuh"

#include <algorithm>
#include <math.h>

namespace kvq {
namespace {

constexpr int kNT = 256;
constexpr int kMaxPairs = 64;
constexpr int kSpan = 18;        // tokens a query CTA may touch
constexpr int kMaxRow = 1024;    // row dims the append handles

struct RopeParams {
    int32_t dim, pairs;
    uint64_t inc[kMaxPairs];
    uint8_t axis[kMaxPairs];
    const int64_t* pos;
    int64_t pos_stride;
    int64_t n;
    // rows
    const void* x;
    int64_t x_stride;
    const int64_t* slots;
    uint8_t* codes;
    float* scales;
    int64_t pool_rows;
    int32_t* err;
    int64_t row_ctas;
    // queries
    const void* qi;
    int64_t qi_tok, qi_head;
    void* qo;
    int64_t qo_tok, qo_head;
    int32_t n_heads;
    int32_t per_tok;   // units of one token
    int32_t per_cta;   // units of one CTA
    Tq4Params enc;
};

__device__ __forceinline__ float2 cos_sin(const RopeParams& p, int64_t tok, int i) {
    const int64_t pos = p.pos[p.axis[i] * p.pos_stride + tok];
    const int64_t phase = (int64_t)((uint64_t)pos * p.inc[i]);
    float s, c;
    sincospif(__ll2float_rn(phase) * 0x1p-63f, &s, &c);
    return make_float2(c, s);
}
// Each product rounded, then one sum: the same bits in every path.
__device__ __forceinline__ float2 turn(float u, float v, float2 cs) {
    return make_float2(__fsub_rn(__fmul_rn(u, cs.x), __fmul_rn(v, cs.y)),
                       __fadd_rn(__fmul_rn(v, cs.x), __fmul_rn(u, cs.y)));
}

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T e[V];
};

// V = elements of 16 bytes (vector units), or 1 (one pair a unit, any strides).
template <typename QT, int V, bool ADJ>
__device__ __forceinline__ void rotate_queries(const RopeParams& p, int64_t cta, float2 (*cs)[kMaxPairs]) {
    const int64_t total = p.n * p.per_tok;
    const int64_t u0 = cta * p.per_cta, u1 = min(u0 + p.per_cta, total);
    const int64_t t0 = u0 / p.per_tok;
    const int n_tok = (int)((u1 - 1) / p.per_tok - t0) + 1;
    for (int i = threadIdx.x; i < n_tok * p.pairs; i += kNT) {
        const int t = i / p.pairs, k = i - t * p.pairs;
        cs[t][k] = cos_sin(p, t0 + t, k);
    }
    __syncthreads();
    const QT* qi = static_cast<const QT*>(p.qi);
    QT* qo = static_cast<QT*>(p.qo);
    constexpr int kPairs = V == 1 ? 1 : (ADJ ? V / 2 : V);   // pairs of a unit
    const int per_head = p.pairs / kPairs;
    const int off0 = (int)(u0 - t0 * p.per_tok);
#pragma unroll 4
    for (int i = threadIdx.x; i < (int)(u1 - u0); i += kNT) {
        const int x = off0 + i, t = x / p.per_tok, y = x - t * p.per_tok;
        const int h = y / per_head, k0 = (y - h * per_head) * kPairs;
        const QT* src = qi + (t0 + t) * p.qi_tok + h * p.qi_head;
        QT* dst = qo + (t0 + t) * p.qo_tok + h * p.qo_head;
        const float2* c = &cs[t][k0];
        if constexpr (V == 1) {
            const int a = ADJ ? 2 * k0 : k0, b = ADJ ? 2 * k0 + 1 : k0 + p.pairs;
            const float2 r = turn(to_f(src[a]), to_f(src[b]), c[0]);
            dst[a] = from_f<QT>(r.x);
            dst[b] = from_f<QT>(r.y);
        } else if constexpr (ADJ) {
            Vec<QT, V> v = *reinterpret_cast<const Vec<QT, V>*>(src + 2 * k0);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                const float2 r = turn(to_f(v.e[2 * j]), to_f(v.e[2 * j + 1]), c[j]);
                v.e[2 * j] = from_f<QT>(r.x);
                v.e[2 * j + 1] = from_f<QT>(r.y);
            }
            *reinterpret_cast<Vec<QT, V>*>(dst + 2 * k0) = v;
        } else {
            Vec<QT, V> a = *reinterpret_cast<const Vec<QT, V>*>(src + k0);
            Vec<QT, V> b = *reinterpret_cast<const Vec<QT, V>*>(src + p.pairs + k0);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float2 r = turn(to_f(a.e[j]), to_f(b.e[j]), c[j]);
                a.e[j] = from_f<QT>(r.x);
                b.e[j] = from_f<QT>(r.y);
            }
            *reinterpret_cast<Vec<QT, V>*>(dst + k0) = a;
            *reinterpret_cast<Vec<QT, V>*>(dst + p.pairs + k0) = b;
        }
    }
}

// One new row by one warp: to shared memory in f32, its trailing dims turned,
// then the codec's row encoder.
template <bool TQ4, typename XT, bool ADJ>
__device__ __forceinline__ void append_row(const RopeParams& p, int64_t tok, float* row, const float* th) {
    const int lane = threadIdx.x & 31;
    const int64_t slot = p.slots[tok];
    if (slot < 0) return;   // a padded row
    if (slot >= p.pool_rows) {
        if (lane == 0 && p.err) atomicCAS(p.err, 0, (int32_t)KVQ_ERR_ARG);
        return;
    }
    const int D = p.enc.D, r0 = D - p.dim;
    const XT* x = static_cast<const XT*>(p.x) + tok * p.x_stride;
    for (int i = lane; i < D; i += 32) row[i] = to_f(x[i]);
    __syncwarp();
    for (int i = lane; i < p.pairs; i += 32) {
        const int a = r0 + (ADJ ? 2 * i : i), b = r0 + (ADJ ? 2 * i + 1 : i + p.pairs);
        const float2 r = turn(row[a], row[b], cos_sin(p, tok, i));
        row[a] = r.x;
        row[b] = r.y;
    }
    __syncwarp();
    float* so = p.scales + slot * p.enc.n_blocks;
    if (!TQ4) {
        kv8_encode_row_from([row](int i) { return row[i]; }, p.enc.n_blocks, p.enc.bd[0], p.enc.bd[1], p.codes + slot * D, so,
                            lane, p.err);
        return;
    }
    int off = 0;
    for (int b = 0; b < p.enc.n_blocks; ++b) {
        const float* xb = row + off;
        uint8_t* ob = p.codes + slot * (D / 2) + off / 2;
        switch (p.enc.bd[b]) {
#define KVQ_CASE(n) \
    case n: tq4_encode_block<n>([xb](int i) { return xb[i]; }, lane, p.enc, b, th, ob, so + b, p.err); break;
            KVQ_POW2_CASES(KVQ_CASE)
#undef KVQ_CASE
            default: break;
        }
        off += p.enc.bd[b];
    }
}

template <bool TQ4, typename XT, typename QT, int V, bool ADJ>
__global__ void __launch_bounds__(kNT) rope_append_kernel(const __grid_constant__ RopeParams p) {
    __shared__ union {
        float2 cs[kSpan][kMaxPairs];
        float row[kNT / 32][kMaxRow];
    } sm;
    __shared__ float th[16];
    launch_dependents();
    grid_dependency_wait();
    if ((int64_t)blockIdx.x >= p.row_ctas) {
        rotate_queries<QT, V, ADJ>(p, (int64_t)blockIdx.x - p.row_ctas, sm.cs);
        return;
    }
    if (TQ4) {
        if (threadIdx.x < 16) th[threadIdx.x] = p.enc.cb.th[threadIdx.x];
        __syncthreads();
    }
    const int warp = threadIdx.x >> 5;
    const int64_t tok = (int64_t)blockIdx.x * (kNT / 32) + warp;
    if (tok < p.n) append_row<TQ4, XT, ADJ>(p, tok, sm.row[warp], th);
}

template <bool TQ4, typename XT, typename QT, int V>
cudaError_t launch_pairs(const RopeParams& p, bool adjacent, int64_t grid, cudaStream_t st) {
    return adjacent ? launch_chained(rope_append_kernel<TQ4, XT, QT, V, true>, (unsigned)grid, kNT, 0, st, p)
                    : launch_chained(rope_append_kernel<TQ4, XT, QT, V, false>, (unsigned)grid, kNT, 0, st, p);
}
template <bool TQ4, typename XT, typename QT>
cudaError_t launch_width(const RopeParams& p, bool adjacent, bool vec, int64_t grid, cudaStream_t st) {
    return vec ? launch_pairs<TQ4, XT, QT, 16 / sizeof(QT)>(p, adjacent, grid, st)
               : launch_pairs<TQ4, XT, QT, 1>(p, adjacent, grid, st);
}
template <bool TQ4>
cudaError_t launch_types(const RopeParams& p, kvq_dtype xt, kvq_dtype qt, bool adjacent, bool vec, int64_t grid,
                         cudaStream_t st) {
    if (xt == KVQ_BF16)
        return qt == KVQ_BF16 ? launch_width<TQ4, __nv_bfloat16, __nv_bfloat16>(p, adjacent, vec, grid, st)
                              : launch_width<TQ4, __nv_bfloat16, float>(p, adjacent, vec, grid, st);
    return qt == KVQ_BF16 ? launch_width<TQ4, float, __nv_bfloat16>(p, adjacent, vec, grid, st)
                          : launch_width<TQ4, float, float>(p, adjacent, vec, grid, st);
}

}  // namespace

cudaError_t launch_rope_append(kvq_format fmt, const kvq_mla_layout& L, const kvq_rope& rope, const void* x,
                               kvq_dtype xt, int64_t x_stride, int64_t n, const int64_t* pos, int64_t pos_stride,
                               const int64_t* slots, const void* qi, kvq_dtype qt, int64_t qi_tok, int64_t qi_head,
                               void* qo, int64_t qo_tok, int64_t qo_head, int32_t n_heads, uint8_t* codes,
                               float* scales, int64_t pool_rows, int32_t* err, cudaStream_t stream) {
    RopeParams p{};
    p.dim = rope.dim;
    p.pairs = rope.dim / 2;
    for (int i = 0; i < p.pairs; ++i) {
        // turns per position as a 64-bit fraction; whole turns drop out
        double f = rope.inv_freq[i] / (2.0 * M_PI);
        if (!(f >= 0.0 && f < 1.0)) f -= floor(f);
        p.inc[i] = f < 1.0 ? (uint64_t)(f * 0x1p64) : 0;
        p.axis[i] = rope.axis[i];
    }
    p.pos = pos;
    p.pos_stride = pos_stride;
    p.n = n;
    p.x = x;
    p.x_stride = x_stride;
    p.slots = slots;
    p.codes = codes;
    p.scales = scales;
    p.pool_rows = pool_rows;
    p.err = err;
    p.row_ctas = x ? (n + kNT / 32 - 1) / (kNT / 32) : 0;
    p.qi = qi;
    p.qi_tok = qi_tok;
    p.qi_head = qi_head;
    p.qo = qo;
    p.qo_tok = qo_tok;
    p.qo_head = qo_head;
    p.n_heads = n_heads;
    p.enc = make_tq4_params(L);
    // 16-byte units where every head's rotary dims start on 16 bytes and split
    // into whole units; one pair at a time otherwise
    const int64_t size = qt == KVQ_BF16 ? 2 : 4, v = 16 / size;
    const bool adjacent = rope.adjacent != 0;
    const bool vec = (adjacent ? rope.dim : p.pairs) % v == 0 && ((uintptr_t)qi | (uintptr_t)qo) % 16 == 0 &&
                     (qi_tok | qi_head | qo_tok | qo_head) % v == 0;
    int64_t q_ctas = 0;
    if (n_heads > 0) {
        const int64_t unit_pairs = !vec ? 1 : adjacent ? v / 2 : v;
        p.per_tok = (int32_t)(n_heads * (p.pairs / unit_pairs));
        // 2 units a thread once that fills the GPU (2048 tokens x 128 heads: 14.3 us,
        // 4 units 15.2, one 17.4)
        int64_t per = 2 * kNT;
        while (per > kNT && n * p.per_tok < per * 304) per /= 2;
        p.per_cta = (int32_t)std::min<int64_t>(per, (int64_t)p.per_tok * (kSpan - 2));
        q_ctas = (n * p.per_tok + p.per_cta - 1) / p.per_cta;
    }
    const int64_t grid = p.row_ctas + q_ctas;
    if (grid == 0) return cudaSuccess;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    return fmt == KVQ_TQ4 ? launch_types<true>(p, xt, qt, adjacent, vec, grid, stream)
                          : launch_types<false>(p, xt, qt, adjacent, vec, grid, stream);
}

}  // namespace kvq
