// gqa_append.cu -- the append of a grouped-query KV8 pool, one launch: the step's
// queries are rotated into place, its keys rotated, keys and values quantized and
// stored in their slots.
//
// Pair i of a head's leading rotary dims turns by pos[axis_i] w_i; angles are kept in
// turns as 64-bit fractions (see rope.cu).  A row of D values gets s = amax / 448 and
// the codes e4m3(x / s), the bytes kv8_encode gives for the rotated f32 row.
//
// What bounds it: memory (queries in and out, keys and values in, codes out).  A group of
// D / 8 threads holds one head's row, 8 elements a thread.  The rows of all tokens are
// numbered through and a CTA takes a run of them; the cos and sin of its tokens are shared
// by their heads, so it tabulates them, while the rows it has asked for are on their way.
// Measured: 12.5 us a call (13 to 14.5 in a replayed graph) for 1999 tokens of 16 query and 2 + 2
// rows of 256 in bf16 (39 MB: 3 TB/s; a plain copy of the queries alone takes 7.9), issue slots 74%
// busy with angles, index arithmetic and the correctly rounded divisions of the codes; 64 tokens of 32 + 8 + 8 heads 4.9 us, the launch's
// latency.
#include "gqa.cuh"

#include <algorithm>
#include <math.h>

namespace kvq {
namespace {

constexpr int kNT = 256;
constexpr int kMaxPairs = 64;
constexpr int kTrips = 4;   // rows a thread group takes at most
constexpr int kSpan = 18;   // tokens a CTA's rows may belong to

struct AppendParams {
    GqaAppendCall c;
    int32_t rot, pairs, shift;
    int64_t pool_rows;
    int64_t total;      // rows of all tokens
    int32_t per_tok;    // of one token
    int32_t per_cta;
    uint32_t ctas;
    uint64_t inc[kMaxPairs];
    uint8_t axis[kMaxPairs];
};

template <typename T>
__device__ __forceinline__ float to_f(T v) { return (float)v; }

// E consecutive elements from any aligned (VEC) or element-aligned address, as they lie in memory.
template <typename T, int E, bool VEC>
struct alignas(16) Elems {
    T e[E];
    __device__ __forceinline__ void load(const T* src) {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(*this) / 16; ++i)
                reinterpret_cast<uint4*>(e)[i] = reinterpret_cast<const uint4*>(src)[i];
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) e[i] = src[i];
        }
    }
    __device__ __forceinline__ void floats(float (&x)[E]) const {
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = to_f(e[i]);
    }
};
template <typename T, int E, bool VEC>
__device__ __forceinline__ void store_elems(T* dst, const float (&x)[E]) {
    if constexpr (VEC) {
        constexpr int V = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < E; i += V) {
            struct alignas(16) { T e[V]; } v;
#pragma unroll
            for (int j = 0; j < V; ++j) v.e[j] = (T)x[i + j];
            *reinterpret_cast<uint4*>(dst + i) = *reinterpret_cast<const uint4*>(&v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) dst[i] = (T)x[i];
    }
}

// CTAs of an SM: 1999 tokens of 16 + 2 + 2 heads of 256 in bf16 take 14.8 us with 3, 13.1 with 5 (a few
// registers spill), 15.4 with 6.  f32 rows take more registers.
template <typename T, int D, bool VEC, bool ADJ>
__global__ void __launch_bounds__(kNT, sizeof(T) == 4 ? 4 : 5) gqa_append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int E = 8, kGroup = D / E, kRows = kNT / kGroup;   // threads of a row, rows a CTA holds at once
    __shared__ float2 table[kSpan][kMaxPairs];
    launch_dependents();
    grid_dependency_wait();
    const GqaAppendCall& a = p.c;
    const int tid = threadIdx.x, t = tid % kGroup, d0 = t * E;
    const int n_kv = a.k ? a.n_kv_heads : 0;
    const int64_t u0 = (int64_t)blockIdx.x * p.per_cta;
    const int count = (int)min((int64_t)p.per_cta, p.total - u0);
    const int64_t t0 = u0 / p.per_tok;
    const int off0 = (int)(u0 - t0 * p.per_tok);   // the run's first row within token t0
    // the thread's rows: row `row` of token t0 + tok, then the one kRows further
    struct Place {
        int tok, row;
        __device__ __forceinline__ void skip(int n, int per_tok) {
            for (row += n; row >= per_tok; row -= per_tok) ++tok;
        }
    };
    const auto source = [&](Place at) {
        return at.row >= 2 * n_kv ? static_cast<const T*>(a.qi) + (t0 + at.tok) * a.qi_token + (int64_t)(at.row - 2 * n_kv) * a.qi_head
               : at.row >= n_kv   ? static_cast<const T*>(a.v) + (t0 + at.tok) * a.v_token + (int64_t)(at.row - n_kv) * a.v_head
                                  : static_cast<const T*>(a.k) + (t0 + at.tok) * a.k_token + (int64_t)at.row * a.k_head;
    };
    const int i0 = tid / kGroup;
    Place start{0, off0};
    start.skip(i0, p.per_tok);
    // asked for before the angles are worked out
    Elems<T, E, VEC> raw[kTrips];
    int64_t slots[kTrips];
    {
        Place at = start;
#pragma unroll
        for (int j = 0; j < kTrips; ++j) {
            slots[j] = -1;
            if (j * kRows + i0 < count) {
                raw[j].load(source(at) + d0);
                if (at.row < 2 * n_kv) slots[j] = a.slots[t0 + at.tok];
            }
            at.skip(kRows, p.per_tok);
        }
    }
    if (p.rot > 0) {
        const int n_tok = (off0 + count - 1) / p.per_tok + 1;
        for (int i = tid; i < n_tok * p.pairs; i += kNT) {
            const int tok = i / p.pairs, k = i - tok * p.pairs;
            const int64_t pos = a.positions[p.axis[k] * a.pos_stride + t0 + tok];
            const int64_t phase = (int64_t)((uint64_t)pos * p.inc[k]);
            float2 cs;
            // half turns in f32 are off by up to 2^-25, which the next term of the angle's sum takes back
            const float h = __ll2float_rn(phase), r = __ll2float_rn(phase - __float2ll_rn(h)) * (float)(M_PI * 0x1p-63);
            sincospif(h * 0x1p-63f, &cs.y, &cs.x);
            table[tok][k] = make_float2(__fmaf_rn(-r, cs.y, cs.x), __fmaf_rn(r, cs.x, cs.y));
        }
        __syncthreads();
    }
    const bool turns = d0 < p.rot, first = ADJ || d0 < p.pairs;
    // every thread of a warp makes every trip: rows past the last are not stored
    Place at = start;
#pragma unroll
    for (int trip = 0; trip < kTrips; ++trip, at.skip(kRows, p.per_tok)) {
        if (trip * kRows >= count) break;
        const bool live = trip * kRows + i0 < count, query = at.row >= 2 * n_kv, value = !query && at.row >= n_kv;
        const int tok = at.tok, h = query ? at.row - 2 * n_kv : value ? at.row - n_kv : at.row;
        float x[E], y[E];
        raw[trip].floats(x);
        if (turns && !value && live) {
            if (ADJ) {
#pragma unroll
                for (int j = 0; j < E; ++j) y[j] = x[j ^ 1];
            } else if (p.pairs % E == 0) {
                Elems<T, E, VEC> other;
                other.load(source(at) + (first ? d0 + p.pairs : d0 - p.pairs));
                other.floats(y);
            } else {
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const int d = d0 + j;
                    y[j] = d >= p.rot ? 0.0f : to_f(source(at)[d < p.pairs ? d + p.pairs : d - p.pairs]);
                }
            }
            // x cos - y sin for the first of a pair, x cos + y sin for the second: each product
            // rounded, then one sum
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int d = d0 + j, k = ADJ ? d / 2 : d < p.pairs ? d : d - p.pairs;
                if (d < p.rot) {
                    const float2 cs = table[tok][k];
                    const bool one = ADJ ? (j & 1) == 0 : d < p.pairs;
                    x[j] = __fadd_rn(__fmul_rn(x[j], cs.x), __fmul_rn(y[j], one ? -cs.y : cs.y));
                }
            }
        }
        __syncwarp();   // a head rotated in place: read before it is written
        if (query && live)
            store_elems<T, E, VEC>(static_cast<T*>(a.qo) + (t0 + tok) * a.qo_token + (int64_t)h * a.qo_head + d0, x);
        if (!__any_sync(kFull, !query)) continue;
        float amax = 0.0f;
        bool bad = false;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            bad |= !(fabsf(x[j]) <= 3.402823466e38f);
            amax = fmaxf(amax, fabsf(x[j]));
        }
#pragma unroll
        for (int o = kGroup / 2; o >= 1; o >>= 1) {
            amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
            bad |= __shfl_xor_sync(kFull, (int)bad, o) != 0;
        }
        if (!live || query) continue;
        const int64_t slot = slots[trip];
        if (slot < 0) continue;   // a padded row
        if (slot >= p.pool_rows) {
            if (t == 0 && a.err) atomicCAS(a.err, 0, (int32_t)KVQ_ERR_ARG);
            continue;
        }
        const float s = __fdiv_rn(amax, 448.0f);
        uint32_t w[2] = {0u, 0u};
        if (s != 0.0f && !bad) {
#pragma unroll
            for (int j = 0; j < E; ++j)
                w[j / 4] |= (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(x[j], s), __NV_SATFINITE, __NV_E4M3) << (8 * (j & 3));
        }
        const int64_t to = (((slot >> p.shift) * a.n_kv_heads + h) << p.shift) + (slot & ((1ll << p.shift) - 1));
        *reinterpret_cast<uint2*>((value ? a.v_codes : a.k_codes) + to * D + d0) = make_uint2(w[0], w[1]);
        // a row that is no number: no codes exist, and its scale says so
        if (t == 0) {
            a.scales[2 * to + value] = bad ? __uint_as_float(0x7fffffffu) : s;
            if (bad && a.err) atomicCAS(a.err, 0, (int32_t)KVQ_ERR_NONFINITE);
        }
    }
}

template <typename T, int D, bool VEC>
cudaError_t launch_pairs(const AppendParams& p, bool adj, cudaStream_t st) {
    return adj ? launch_chained(gqa_append_kernel<T, D, VEC, true>, p.ctas, kNT, 0, st, p)
               : launch_chained(gqa_append_kernel<T, D, VEC, false>, p.ctas, kNT, 0, st, p);
}
template <typename T, int D>
cudaError_t launch_width(const AppendParams& p, bool vec, bool adj, cudaStream_t st) {
    return vec ? launch_pairs<T, D, true>(p, adj, st) : launch_pairs<T, D, false>(p, adj, st);
}
template <typename T>
cudaError_t launch_dim(const AppendParams& p, bool vec, bool adj, cudaStream_t st) {
    switch (p.c.head_dim) {
        case 64: return launch_width<T, 64>(p, vec, adj, st);
        case 128: return launch_width<T, 128>(p, vec, adj, st);
        default: return launch_width<T, 256>(p, vec, adj, st);
    }
}

}  // namespace

cudaError_t launch_gqa_append(const GqaAppendCall& c, cudaStream_t stream) {
    AppendParams p{};
    p.c = c;
    p.rot = c.rope ? c.rope->dim : 0;
    p.pairs = p.rot / 2;
    for (int i = 0; i < p.pairs; ++i) {
        // turns per position as a 64-bit fraction; whole turns drop out
        double f = c.rope->inv_freq[i] / (2.0 * M_PI);
        if (!(f >= 0.0 && f < 1.0)) f -= floor(f);
        p.inc[i] = f < 1.0 ? (uint64_t)(f * 0x1p64) : 0;
        p.axis[i] = c.rope->axis[i];
    }
    while ((1 << p.shift) < c.page_rows) ++p.shift;
    p.pool_rows = (int64_t)c.n_pages << p.shift;
    p.per_tok = (c.k ? 2 * c.n_kv_heads : 0) + c.n_heads;
    p.total = c.n * p.per_tok;
    // up to 4 rows a thread group once that fills the GPU
    const int64_t rows = kNT * 8 / c.head_dim;
    int64_t per = kTrips * rows;
    while (per > rows && p.total < per * 304) per /= 2;
    p.per_cta = (int32_t)std::min<int64_t>(per, (int64_t)p.per_tok * (kSpan - 2));
    const int64_t ctas = (p.total + p.per_cta - 1) / p.per_cta;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    p.ctas = (uint32_t)ctas;
    // 16-byte accesses where every row starts on 16 bytes
    const int64_t v = c.dtype == KVQ_BF16 ? 8 : 4;
    uintptr_t where = 0;
    int64_t strides = 0;
    if (c.k) {
        where |= (uintptr_t)c.k | (uintptr_t)c.v;
        strides |= c.k_token | c.k_head | c.v_token | c.v_head;
    }
    if (c.n_heads > 0) {
        where |= (uintptr_t)c.qi | (uintptr_t)c.qo;
        strides |= c.qi_token | c.qi_head | c.qo_token | c.qo_head;
    }
    const bool vec = where % 16 == 0 && strides % v == 0, adj = c.rope && c.rope->adjacent != 0;
    return c.dtype == KVQ_BF16 ? launch_dim<__nv_bfloat16>(p, vec, adj, stream) : launch_dim<float>(p, vec, adj, stream);
}

}  // namespace kvq
