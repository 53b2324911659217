// gqa_append.cu -- the append of a grouped-query KV8 pool, one launch: the step's
// queries are rotated into place, its keys rotated, keys and values quantized and
// stored in their slots.
//
// Pair i of a head's leading rotary dims turns by pos[axis_i] w_i; angles are kept in
// turns as 64-bit fractions (see rope.cu).  A row of D values gets s = amax / 448 and
// the codes e4m3(x / s), the bytes kv8_encode gives for the rotated f32 row.
//
// What bounds it: memory (queries in and out, keys and values in, codes out).  A CTA
// serves one token: a group of T threads holds one head's row, 16 bytes or two times
// 16 a thread, and runs through the token's heads with the same dims, so a thread works
// out its dims' cos and sin once.  Keys and values come first: their chain (load,
// rotate, amax over the group, codes) is the longest.
#include "gqa.cuh"

#include <math.h>

namespace kvq {
namespace {

constexpr int kNT = 256;
constexpr int kMaxPairs = 64;

struct AppendParams {
    GqaAppendCall c;
    int32_t rot, pairs, shift;
    int64_t pool_rows;
    uint64_t inc[kMaxPairs];
    uint8_t axis[kMaxPairs];
};

template <typename T>
__device__ __forceinline__ float to_f(T v) { return (float)v; }

// E consecutive elements from or to any aligned (VEC) or element-aligned address.
template <typename T, int E, bool VEC>
__device__ __forceinline__ void load_elems(float (&x)[E], const T* src) {
    if constexpr (VEC) {
        constexpr int V = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < E; i += V) {
            struct alignas(16) { T e[V]; } v;
            *reinterpret_cast<uint4*>(&v) = *reinterpret_cast<const uint4*>(src + i);
#pragma unroll
            for (int j = 0; j < V; ++j) x[i + j] = to_f(v.e[j]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = to_f(src[i]);
    }
}
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

// E elements a thread: 8, a row of D by D / 8 threads.
template <typename T, int D, bool VEC, bool ADJ>
__global__ void __launch_bounds__(kNT) gqa_append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int E = 8, T_ = D / E, kRows = kNT / T_;   // threads of a row, rows a CTA holds at once
    launch_dependents();
    grid_dependency_wait();
    const GqaAppendCall& a = p.c;
    const int tid = threadIdx.x, t = tid % T_, d0 = t * E;
    const int64_t tok = blockIdx.x;
    // this thread's cos and sin: of pair (d / 2) or (d mod pairs), with the partner's sign
    float cs[E], sn[E];
    const bool turns = d0 < p.rot;
    if (turns) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int d = d0 + i, k = min(ADJ ? d / 2 : (d < p.pairs ? d : d - p.pairs), p.pairs - 1);
            if (ADJ && (i & 1)) {
                cs[i] = cs[i - 1];
                sn[i] = -sn[i - 1];
            } else {
                const int64_t pos = a.positions[p.axis[k] * a.pos_stride + tok];
                const int64_t phase = (int64_t)((uint64_t)pos * p.inc[k]);
                sincospif(__ll2float_rn(phase) * 0x1p-63f, &sn[i], &cs[i]);
                // x cos - y sin for the first of a pair, x cos + y sin for the second
                if (ADJ || d < p.pairs) sn[i] = -sn[i];
            }
            if (d >= p.rot) {
                cs[i] = 1.0f;
                sn[i] = 0.0f;
            }
        }
    }
    const int64_t slot = a.k ? a.slots[tok] : -1;
    const bool store = slot >= 0 && slot < p.pool_rows;
    if (a.k && slot >= p.pool_rows && tid == 0 && a.err) atomicCAS(a.err, 0, (int32_t)KVQ_ERR_ARG);
    const int n_kv = a.k ? a.n_kv_heads : 0, n_rows = 2 * n_kv + a.n_heads;
    const int64_t page_row = store ? ((slot >> p.shift) * a.n_kv_heads << p.shift) + (slot & ((1ll << p.shift) - 1)) : 0;
    // every thread of a warp makes every trip: rows past the last are not stored
    for (int row0 = 0; row0 < n_rows; row0 += kRows) {
        const int row = row0 + tid / T_;
        const bool live = row < n_rows, query = row >= 2 * n_kv, value = !query && row >= n_kv;
        const int h = query ? row - 2 * n_kv : value ? row - n_kv : row;
        const T* src = query ? static_cast<const T*>(a.qi) + tok * a.qi_token + (int64_t)h * a.qi_head
                       : value ? static_cast<const T*>(a.v) + tok * a.v_token + (int64_t)h * a.v_head
                               : static_cast<const T*>(a.k) + tok * a.k_token + (int64_t)h * a.k_head;
        float x[E], y[E];
        if (live) load_elems<T, E, VEC>(x, src + d0);
        if (live && turns && !value) {
            if (ADJ) {
#pragma unroll
                for (int i = 0; i < E; ++i) y[i] = x[i ^ 1];
            } else if (p.pairs % E == 0) {
                load_elems<T, E, VEC>(y, src + (d0 < p.pairs ? d0 + p.pairs : d0 - p.pairs));
            } else {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const int d = d0 + i;
                    y[i] = d >= p.rot ? 0.0f : to_f(src[d < p.pairs ? d + p.pairs : d - p.pairs]);
                }
            }
            // each product rounded, then one sum
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (d0 + i < p.rot) x[i] = __fadd_rn(__fmul_rn(x[i], cs[i]), __fmul_rn(y[i], sn[i]));
        }
        __syncwarp();   // a head rotated in place: read before it is written
        if (query) {
            if (live) store_elems<T, E, VEC>(static_cast<T*>(a.qo) + tok * a.qo_token + (int64_t)h * a.qo_head + d0, x);
        }
        float amax = 0.0f;
        bool bad = false;
        if (live && !query) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                bad |= !(fabsf(x[i]) <= 3.402823466e38f);
                amax = fmaxf(amax, fabsf(x[i]));
            }
        }
        if (row0 < 2 * n_kv) {   // alike for the whole CTA
#pragma unroll
            for (int o = T_ / 2; o >= 1; o >>= 1) {
                amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
                bad |= __shfl_xor_sync(kFull, (int)bad, o) != 0;
            }
            if (live && !query && store) {
                const float s = __fdiv_rn(amax, 448.0f);
                uint32_t w[2] = {0u, 0u};
                if (s != 0.0f && !bad) {
#pragma unroll
                    for (int i = 0; i < E; ++i)
                        w[i / 4] |= (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(x[i], s), __NV_SATFINITE, __NV_E4M3)
                                    << (8 * (i & 3));
                }
                const int64_t at = page_row + ((int64_t)h << p.shift);
                *reinterpret_cast<uint2*>((value ? a.v_codes : a.k_codes) + at * D + d0) = make_uint2(w[0], w[1]);
                // a row that is no number: no codes exist, and its scale says so
                if (t == 0) {
                    a.scales[2 * at + value] = bad ? __uint_as_float(0x7fffffffu) : s;
                    if (bad && a.err) atomicCAS(a.err, 0, (int32_t)KVQ_ERR_NONFINITE);
                }
            }
        }
    }
}

template <typename T, int D, bool VEC>
cudaError_t launch_pairs(const AppendParams& p, bool adj, cudaStream_t st) {
    return adj ? launch_chained(gqa_append_kernel<T, D, VEC, true>, (unsigned)p.c.n, kNT, 0, st, p)
               : launch_chained(gqa_append_kernel<T, D, VEC, false>, (unsigned)p.c.n, kNT, 0, st, p);
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
    if (c.n > 0x7fffffff) return cudaErrorInvalidConfiguration;
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
