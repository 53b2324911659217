// gqa_tc.cu -- attention over paged KV8 keys and values where a sequence brings many
// query vectors to a kv head (prompt chunks, decoder prompts over an encoder's states,
// wide windows): tiles of 128 vectors on the tensor cores.
//
//   S = Q C_k^T (128 vectors x 128 rows), P = 2^(z - R) s_v, O += P C_v
// with z = S s_k sm log2(e), the codes in f16 (exact), f32 accumulators in tensor memory.
//
// What bounds it: the chain of a step (scores, softmax, weights into tensor memory, products), which
// one tile can't overlap with itself: tensor memory holds two tiles' scores and contexts and no more.
// So two CTAs share an SM, one's softmax beside the other's products, and the weights go
// into the second product from tensor memory, over the scores they came from, instead of
// through shared memory.  512 bf16 tokens of 32 heads (8 of keys) of 128 on 8704 rows: 116 us, 611
// TFLOP/s; at 133 us the tensor pipe was 24% busy, shared memory 43%, issue slots 33%.
// A step takes one CTA some 6,200 cycles: 3,200 the softmax, 2,400 the products (issuing, waiting for the
// weights' product and for the scores).  Slower (of 133 us then): scores of 64 rows in two buffers (157);
// the next scores loaded ahead, with more registers for the softmax and fewer for the converters
// (154); eight softmax warps, half of the rows each (215: 80 registers).  Beside the steps a CTA spends
// some 10,000 cycles on finding its place (by bisection over the tiles 17,000), 4,000 on the first queries
// and as many on each tile's outputs.
//   * warps 0-3: softmax, a vector a thread, so maxima and sums need no exchange; 32 scores at
//     a time are loaded, turned into weights and stored over the first half of the scores'
//     place (f32 queries: two f16 halves, over the whole place);
//   * warps 4-7: codes to f16, in the layout of 128-byte swizzled rows, which the first
//     product reads with dims along K and the second with rows along K; keys and values are asked
//     for in turn, each as soon as the other is stored;
//   * a lane of warp 0 issues the products: between its weights and the next scores the
//     softmax has nothing to do (a ninth warp for it left 96 registers a thread, which
//     spilled, and one of the converters' was missed there: 155 us).
//
// Numbers.  Queries as in gqa_attn.cu (bf16 exactly, f32 in two f16 halves).  R is an
// integer per vector, max(z + log2 s_v) - 8 when it is set (f32 queries: 12), and at least max(z) - 100,
// which rows of zero values leave it at; it rises when a weight passes 60000, and then what has been
// summed is brought to it by a power of two.  bf16
// queries: weights in one f16 (2^-11 of themselves, down to 2^-22 of the largest).
// f32 queries: in two (2^-22); products of the small halves come first, since each rounds the sum
// so far.  Every 256 steps (f32 queries: 8) the accumulators, which round
// towards zero, go to totals in the workspace.  Rows that are no numbers as in gqa_attn.cu.
#include "gqa_common.cuh"

#include <algorithm>

namespace kvq {
namespace {

using namespace tc;

constexpr int kM = 128, kN = 128, kOv = 3;
constexpr int kSoft = 128, kConv = 128, kNT = kSoft + kConv;
constexpr float kNone = -3.402823466e38f;
using Walk = GqaWalk<kM, kN, kOv, 4>;   // 128 vectors on 8000 rows: 37 us at least 1, 30 at 4, 39 at 8

template <int D, int QP>
struct Cfg {
    static constexpr int kChunks = D / 64;                      // of 64 dims, 128 rows x 128 bytes each
    static constexpr uint32_t kChunk = 128 * 128;
    static constexpr uint32_t kOffQ = 0, kOffK = QP * kChunks * kChunk, kOffV = kOffK + kChunks * kChunk;
    static constexpr uint32_t kOffMisc = kOffV + kChunks * kChunk;
    static constexpr int kCols = D == 256 ? 512 : 256;          // tensor memory: scores and weights, context
    static constexpr int kColO = 128;
    // steps between additions to the totals: 8 QP products a step, each off by up to 2^-24 of the
    // sum towards zero, add up to 8e-6 (f32) and 1.2e-4 of it
    static constexpr int kFlush = QP == 2 ? 8 : 256;
    static constexpr int kCtas = D == 256 || (D == 128 && QP == 2) ? 1 : 2;   // an SM
};
enum { kBarK, kBarS, kBarV, kBarO, kBarDone, kBarNever, kBars };

struct Misc {
    float sk[2][kN], sv[2][kN];
    float sv_top[2][kN / 32];   // largest of 32 rows
    float qs[kM];
    float ref_tot[kM], sum_tot[kM];   // of the totals
    uint64_t bars[kBars];
    int64_t part[2 * (kNT / 32) + 2];
    Walk walk;
    GqaSegment seg;
    uint32_t tmem;
    int more, abort;
};

__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc));
}

// Columns of weights of scores 16 i ..: over the first half of the scores' place, or (two halves)
// over all of it.
template <int QP>
__device__ __forceinline__ constexpr uint32_t weight_col(int i) { return QP == 1 ? 8u * i : 16u * i; }
constexpr int kC = 32;   // scores taken at a time
template <int QP>
constexpr int kWords = QP * kC / 2;   // of so many weights: first halves of 16, second halves of 16, ...

__device__ __forceinline__ void load_weights(uint32_t t, uint32_t (&v)[16]) { tmem_ld16(t, v); }
__device__ __forceinline__ void load_weights(uint32_t t, uint32_t (&v)[32]) { tmem_ld32(t, v); }
__device__ __forceinline__ void store_weights(uint32_t t, const uint32_t (&v)[16]) { tmem_st16(t, v); }
__device__ __forceinline__ void store_weights(uint32_t t, const uint32_t (&v)[32]) { tmem_st32(t, v); }

// The softmax's waits, for a phase of each of two barriers at once: polls without suspending (a suspended
// lane woke some 800 cycles late, with every product of the CTA behind it), and looks at the abort
// flag only when the first fails: with the converters' stores in the queue a read of shared memory
// takes some 150 cycles.
__device__ __forceinline__ bool mbar_spin(uint64_t* x, uint32_t px, uint64_t* y, uint32_t py, volatile int* abort_flag,
                                          long long limit) {
    const uint32_t a = smem_u32(x), b = smem_u32(y);
    for (long long i = 0; i < 16 * limit; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p, q;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
            " mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %4;\n and.pred p, p, q;\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(a), "r"(px), "r"(b), "r"(py)
            : "memory");
        if (ok) return true;
        if ((i & 63) == 0 && *abort_flag) return false;
    }
    *abort_flag = 1;
    return false;
}
__device__ __forceinline__ bool mbar_spin(uint64_t* bar, uint32_t parity, volatile int* abort_flag, long long limit) {
    const uint32_t a = smem_u32(bar);
    for (long long i = 0; i < 16 * limit; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(a), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((i & 63) == 0 && *abort_flag) return false;
    }
    *abort_flag = 1;
    return false;
}

// x 2^d, d whole and at most 0: 2^d alone may lie below f32 where the product does not (sums of weights before
// the values' scales, under a reference that a large scale raised).
__device__ __forceinline__ float times_2(float x, float d) {
    const float h = truncf(0.5f * d);
    return x * ex2(h) * ex2(d - h);
}

// A vector's reference raised for chunk j of a step (see the file's head), by a whole warp: its weights of
// the chunks before (tm: its scores) and its context (to) are brought to the new one, which is returned.
template <int D, int QP>
__device__ __forceinline__ float raise(const Misc& sm, uint32_t tm, uint32_t to, int j, int st, float qs, float R, bool lift,
                                       int32_t visible, bool context) {
    uint32_t s[kC];
    tmem_ld32(tm + kC * j, s);
    tmem_wait_ld();
    float y = kNone, zm = kNone;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
        const float sv = fabsf(sm.sv[st][kC * j + i]), z = __uint_as_float(s[i]) * (sm.sk[st][kC * j + i] * qs);
        if (i < visible) {
            zm = fmaxf(zm, z);
            if (sv > 0.0f) y = fmaxf(y, z + __log2f(sv));
        }
    }
    float n = R;
    if (lift) n = fmaxf(R, ceilf(fmaxf(y - (QP == 1 ? 8.0f : 12.0f), zm - 100.0f)));
    if (!(n >= kNone)) n = kNone;   // no score but -inf
    const float a = n == R ? 1.0f : ex2(R - n);
    // in f32: the factor may lie below f16's range where the weights, up to 2^16 of the old reference, stay in it
#pragma unroll 1
    for (int k = 0; k < j; ++k) {
        uint32_t w[kWords<QP>];
        load_weights(tm + weight_col<QP>(k * (kC / 16)), w);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < kC; c += 2) {
            const int at = QP * 8 * (c / 16) + c % 16 / 2;
            float2 x = unpack_half2(w[at]);
            if constexpr (QP == 2) {   // the halves' sum is exact: 22 bits
                const float2 y = unpack_half2(w[8 + at]);
                x = make_float2(x.x + y.x, x.y + y.y);
            }
            x = make_float2(x.x * a, x.y * a);
            w[at] = pack_half2(x.x, x.y);
            if constexpr (QP == 2) {
                const float2 y = unpack_half2(w[at]);
                w[8 + at] = pack_half2(x.x - y.x, x.y - y.y);
            }
        }
        store_weights(tm + weight_col<QP>(k * (kC / 16)), w);
    }
    if (context) {
#pragma unroll 1
        for (int k = 0; k < D / 32; ++k) {
            uint32_t o[32];
            tmem_ld32(to + 32 * k, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
            tmem_st32(to + 32 * k, o);
        }
    }
    tmem_wait_st();
    return n;
}

// Scores kC j .. of a step to weights; their sum before the values' scales.  PART: some are hidden from
// some vector.
template <int QP, bool PART>
__device__ __forceinline__ float weights(const Misc& sm, const uint32_t (&s)[kC], int j, int st, float qs, float R,
                                         int32_t visible, uint32_t (&pk)[kWords<QP>], float* most) {
    const F2 qs2 = f2(qs, qs), r2 = f2(-R, -R);
    F2 sum[2] = {f2(0.0f, 0.0f), f2(0.0f, 0.0f)};
#pragma unroll
    for (int q = 0; q < kC / 4; ++q) {
        const float4 k4 = *reinterpret_cast<const float4*>(&sm.sk[st][kC * j + 4 * q]);
        const float4 v4 = *reinterpret_cast<const float4*>(&sm.sv[st][kC * j + 4 * q]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = 4 * q + 2 * h, at = QP * 8 * (c / 16) + c % 16 / 2;
            const F2 b = mul2(h == 0 ? f2(k4.x, k4.y) : f2(k4.z, k4.w), qs2);
            const float2 t = unpack(fma2(f2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), b, r2));
            float2 p = make_float2(ex2(t.x), ex2(t.y));
            if (PART) {
                if (c >= visible) p.x = 0.0f;
                if (c + 1 >= visible) p.y = 0.0f;
            }
            const F2 pp = f2(p.x, p.y);
            sum[h] = add2(sum[h], pp);
            float2 w = unpack(mul2(pp, h == 0 ? f2(v4.x, v4.y) : f2(v4.z, v4.w)));
            if (PART) {   // a hidden row's scale may be no number
                if (c >= visible) w.x = 0.0f;
                if (c + 1 >= visible) w.y = 0.0f;
            }
            const uint32_t hi = pack_half2(w.x, w.y);
            pk[at] = hi;
            if constexpr (QP == 2) {
                *most = fmaxf(*most, fmaxf(fabsf(w.x), fabsf(w.y)));
                const float2 x = unpack_half2(hi);
                pk[8 + at] = pack_half2(w.x - x.x, w.y - x.y);
            }
        }
    }
    const float2 u = unpack(add2(sum[0], sum[1]));
    return u.x + u.y;
}

// The codes of one step's keys or values as a converter warp holds them: 32 rows, 16 bytes a lane
// and load, D / 16 lanes a row.  Lanes of odd chunks (of 64 dims) take the neighbouring row, so
// that the f16 of 8 lanes go to different banks.
template <int D>
struct Codes {
    static constexpr int kLanes = D / 16, kAt = 32 / kLanes, kLoads = 32 / kAt;   // lanes of a row, rows a load, loads
    uint4 v[kLoads];
    static __device__ __forceinline__ int row(int lane) { return (lane / kLanes) ^ ((lane % kLanes / 4) & 1); }
    // at: the pool rows that hold rows 0 .. 15 and 16 .. 31 (pages hold at least 16 rows), -1: none of them
    // is seen
    __device__ __forceinline__ void load(const uint8_t* base, const int64_t (&at)[2], int lane) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const uint8_t* src = base + at[g] * D + row(lane) * D + 16 * (lane % kLanes);
#pragma unroll
            for (int i = 0; i < kLoads / 2; ++i)
                v[g * (kLoads / 2) + i] = at[g] >= 0 ? ldg16(src + i * kAt * D) : make_uint4(0u, 0u, 0u, 0u);
        }
    }
    // to f16 in swizzled rows; region: the operand's first chunk, at the warp's first row
    __device__ __forceinline__ void store(unsigned char* region, int lane) const {
        const int q = lane % 4, c = lane % kLanes / 4, r0 = row(lane);
        unsigned char* at = region + c * (128 * 128) + r0 * 128;
        // row i kAt + r0 of the warp's: its place in the swizzle repeats every 8 rows
        constexpr int kTurn = kAt >= 8 ? 1 : 8 / kAt;
        uint32_t lo_at[kTurn], hi_at[kTurn];
#pragma unroll
        for (int t = 0; t < kTurn; ++t) {
            lo_at[t] = (uint32_t)(((2 * q) ^ (t * kAt + r0)) & 7) << 4;
            hi_at[t] = lo_at[t] ^ 16u;
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            uint4 lo, hi;
            e4m3x4_to_half2x2(v[i].x, lo.x, lo.y);
            e4m3x4_to_half2x2(v[i].y, lo.z, lo.w);
            e4m3x4_to_half2x2(v[i].z, hi.x, hi.y);
            e4m3x4_to_half2x2(v[i].w, hi.z, hi.w);
            *reinterpret_cast<uint4*>(at + i * kAt * 128 + lo_at[i % kTurn]) = lo;
            *reinterpret_cast<uint4*>(at + i * kAt * 128 + hi_at[i % kTurn]) = hi;
        }
    }
    // NaN codes replaced; true for the lane whose row holds one
    __device__ __forceinline__ bool mend(int lane) {
        uint32_t rows = 0u;   // rows with one, as this lane sees them
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            uint32_t* w = reinterpret_cast<uint32_t*>(&v[i]);
            bool bad = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t nan = (((w[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
                bad |= nan != 0u;
                w[k] ^= nan;
            }
            if (bad) rows |= 1u << (i * kAt + row(lane));
        }
        return (__reduce_or_sync(kFull, rows) >> lane) & 1u;
    }
};

// Queries of the tile to f16: a warp takes 16 vectors, a lane 16 bytes of one at a time, all asked for at
// once.
template <int D, int QP, typename QT>
__device__ __forceinline__ void load_queries(const GqaParams& p, const GqaSegment& g, Misc& sm, unsigned char* sq) {
    constexpr int V = 16 / sizeof(QT), kLanes = D / V, kAt = 32 / kLanes;   // elements a lane, lanes a vector, vectors a load
    constexpr int kVecs = kM / (kNT / 32), kLoads = kVecs / kAt;
    const int lane = threadIdx.x & 31, r0 = (threadIdx.x >> 5) * kVecs + lane / kLanes, d = lane % kLanes * V;
    struct alignas(16) Piece {
        QT e[V];
    } v[kLoads];
    int32_t tok = (int32_t)((uint32_t)(g.vec0 + r0) / (uint32_t)p.group), rem = g.vec0 + r0 - tok * p.group;
    const QT* src = static_cast<const QT*>(p.q) + (g.q0 * p.n_heads + g.h * p.group) * (int64_t)D + d;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        *reinterpret_cast<uint4*>(&v[i]) =
            r0 + i * kAt < g.vecs ? ldg16(src + ((int64_t)tok * p.n_heads + rem) * D) : make_uint4(0u, 0u, 0u, 0u);
        for (rem += kAt; rem >= p.group; rem -= p.group) ++tok;
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int r = r0 + i * kAt;
        float amax = 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k) amax = fmaxf(amax, fabsf((float)v[i].e[k]));
#pragma unroll
        for (int o = kLanes / 2; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
        const int e = max((int)(__float_as_uint(amax) >> 23) - 127 - 14, -110);
        const float up = __uint_as_float((uint32_t)(127 - e) << 23);
        if (d == 0) sm.qs[r] = query_scale(p.sm_scale, e, amax);
        uint32_t hi[V / 2], lo[V / 2];
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
            const float a = (float)v[i].e[2 * k] * up, b = (float)v[i].e[2 * k + 1] * up;
            hi[k] = pack_half2(a, b);
            const float2 h = unpack_half2(hi[k]);
            lo[k] = pack_half2(a - h.x, b - h.y);
        }
        unsigned char* at = sq + (d / 64) * (128 * 128) + sw128(r, 2 * (d % 64));
        if constexpr (QP == 1) {
            *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        } else {
            *reinterpret_cast<uint2*>(at) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(at + (D / 64) * (128 * 128)) = make_uint2(lo[0], lo[1]);
        }
    }
}

template <typename QT>
__device__ __forceinline__ void store8(QT* dst, const float (&x)[8]) {
    if constexpr (sizeof(QT) == 4) {
        reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
            w[k] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// State of a cut tile's vector: (log2 of its sum of 2^z, context over that sum).
template <int D, int QP, typename QT>
__global__ void __launch_bounds__(kNT, (Cfg<D, QP>::kCtas)) gqa_tc_kernel(const __grid_constant__ GqaParams p) {
    extern __shared__ __align__(1024) unsigned char raw[];
    using C = Cfg<D, QP>;
    Misc& sm = *reinterpret_cast<Misc*>(raw + C::kOffMisc);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();
    if (tid == 0) p.cuts[blockIdx.x].count = 0;
    if (p.n_seq <= Walk::kFew) {
        if (warp == 0) {
            Walk walk;
            const bool any = walk.start_few(p, blockIdx.x, gridDim.x);
            if (lane == 0) {
                sm.walk = walk;
                sm.more = any && walk.get(p, sm.seg);
            }
        }
    } else {
        Walk walk;
        const bool any = walk.template start_many<kNT>(p, blockIdx.x, gridDim.x, sm.part, sm.part + 2 * (kNT / 32));
        if (tid == 0) {
            sm.walk = walk;
            sm.more = any && walk.get(p, sm.seg);
        }
    }
    __syncthreads();
    if (!sm.more) return;
    if (smem_u32(raw) & 1023u) {   // the swizzle counts on it
        if (tid == 0) set_err(p.err, KVQ_ERR_DEVICE);
        return;
    }
    if (warp == 4) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem)),
                     "r"(C::kCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid == 0) {
        for (int i = 0; i < kBars; ++i)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(&sm.bars[i])),
                         "r"(i == kBarK || i == kBarV ? 128u : 1u));
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sm.abort = 0;
    }
    tc_before();
    __syncthreads();
    tc_after();
    launch_dependents();   // a kernel that allocates tensor memory may come now: this CTA has its own
    const uint32_t tmem = sm.tmem;
    volatile int* abort_flag = &sm.abort;
    if (p.stall_polls > 0) {
        if (tid == 0) mbar_wait(&sm.bars[kBarNever], 0, abort_flag, p.stall_polls);
        __syncthreads();
    }
    const GqaSegment& seg = sm.seg;
    uint32_t it = 0;       // steps so far: the barriers' phases
    uint32_t tiles = 0;
    for (;; ++tiles) {
        if (sm.abort) break;   // alike for all: nothing raises it here
        const int u0 = seg.u0, n_steps = seg.limit > u0 * kN ? min(seg.u1 - u0, (seg.limit - u0 * kN + kN - 1) / kN) : 0;
        const int32_t all = gqa_limit(p, seg, seg.vec0);   // rows that all vectors see
        load_queries<D, QP, QT>(p, seg, sm, raw + C::kOffQ);
        fence_async_smem();
        __syncthreads();
        if (warp < 4) {
            // ---- softmax: vector tid -----------------------------------------------
            const int32_t lim = gqa_limit(p, seg, seg.vec0 + min(tid, seg.vecs - 1));
            const float qs = sm.qs[tid];
            const uint32_t tm = tmem + ((uint32_t)(warp * 32) << 16);
            float R = kNone, l = 0.0f;   // reference and sum
            // accumulators to the totals: first: they start there
            auto flush = [&](bool first) {
                float4* tot = reinterpret_cast<float4*>(p.ws_tot) + (int64_t)blockIdx.x * (D / 4) * kM + tid;
                const float Rt = first ? kNone : sm.ref_tot[tid], lt = first ? 0.0f : sm.sum_tot[tid];
                const float n = fmaxf(Rt, R), a = first ? 0.0f : ex2(Rt - n), b = ex2(R - n);
#pragma unroll 1
                for (int k = 0; k < D / 32; ++k) {
                    uint32_t o[32];
                    tmem_ld32(tm + C::kColO + 32 * k, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float4 v = first ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : tot[(8 * k + i) * kM];
                        v.x = v.x * a + __uint_as_float(o[4 * i]) * b;
                        v.y = v.y * a + __uint_as_float(o[4 * i + 1]) * b;
                        v.z = v.z * a + __uint_as_float(o[4 * i + 2]) * b;
                        v.w = v.w * a + __uint_as_float(o[4 * i + 3]) * b;
                        tot[(8 * k + i) * kM] = v;
                    }
                }
                sm.sum_tot[tid] = times_2(lt, Rt - n) + times_2(l, R - n);
                sm.ref_tot[tid] = n;
                l = 0.0f;
            };
            // the products, by one lane
            constexpr uint32_t kIdescS = idesc_f16(kM, kN, false, false), kIdescO = idesc_f16(kM, D, false, true);
            constexpr uint32_t kStep = C::kChunk >> 4;
            auto issue_scores = [&](int s) {
                // the weights of the step before lie over these scores
                if (s > 0 && !mbar_spin(&sm.bars[kBarO], ((it + s) & 1u) ^ 1u, abort_flag, p.wait_limit)) return;
                tc_after();
                const uint64_t dq = umma_desc(smem_u32(raw + C::kOffQ), 16, 1024);
                const uint64_t dk = umma_desc(smem_u32(raw + C::kOffK), 16, 1024);
#pragma unroll
                for (int q = QP - 1; q >= 0; --q)   // the small halves first: each product rounds the sum so far
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const uint32_t at = (i / 4) * kStep + 2 * (i % 4);
                        umma_f16(tmem, dq + q * C::kChunks * kStep + at, dk + at, kIdescS, q < QP - 1 || i > 0);
                    }
                umma_commit(&sm.bars[kBarS]);
            };
            auto issue_context = [&](int s) {
                tc_after();
                const uint64_t dv = umma_desc(smem_u32(raw + C::kOffV), C::kChunk, 1024);
#pragma unroll
                for (int q = QP - 1; q >= 0; --q)
#pragma unroll
                    for (int i = 0; i < kN / 16; ++i)
                        umma_f16_ts(tmem + C::kColO, tmem + weight_col<QP>(i) + 8 * q, dv + 128 * i, kIdescO,
                                    s % C::kFlush != 0 || q < QP - 1 || i > 0);
                umma_commit(&sm.bars[kBarO]);
            };
            if (tid == 0 && n_steps > 0 && mbar_spin(&sm.bars[kBarK], it & 1u, abort_flag, p.wait_limit)) issue_scores(0);
            __syncwarp();
            bool ok = true;
            for (int s = 0; s < n_steps; ++s) {
                const uint32_t ph = (it + s) & 1u;
                const int st = (int)ph;
                // (the scales too: their writers arrived on kBarK, which the issuing lane waited for.  Not
                // waited for here: the next keys' arrival could be the phase after, seen as not yet)
                ok = __all_sync(kFull, mbar_spin(&sm.bars[kBarS], ph, abort_flag, p.wait_limit));
                if (ok) {
                    tc_after();
                    if (s > 0 && s % C::kFlush == 0) flush(s == C::kFlush);
                    const int32_t row0 = (u0 + s) * kN;
                    const bool partly = row0 + kN > all, context = s % C::kFlush != 0;
                    // a reference that had to rise takes its scores again (kept in registers meanwhile, they
                    // would be spilled every time)
#pragma unroll 1
                    for (int j = 0, pass = 0; j < kN / kC;) {
                        const int32_t visible = partly ? min(max(lim - row0 - kC * j, 0), kC) : kC;
                        uint32_t now[kC], pk[kWords<QP>];
                        tmem_ld32(tm + kC * j, now);
                        const float svt = sm.sv_top[st][j];
                        tmem_wait_ld();
                        float sum, most = 0.0f;
                        if (partly) sum = weights<QP, true>(sm, now, j, st, qs, R, visible, pk, &most);
                        else sum = weights<QP, false>(sm, now, j, st, qs, R, kC, pk, &most);
                        // one half: the sum and the scales bound the weights (references leave the room, a false
                        // alarm only costs time); two: the weights themselves
                        if (QP == 1) most = sum * svt;
                        const bool lift = (R == kNone && visible > 0) || !(most <= 60000.0f) || !(sum <= 0x1p110f);
                        if (pass == 0 && __any_sync(kFull, lift)) {
                            const float n = raise<D, QP>(sm, tm, tm + C::kColO, j, st, qs, R, lift, visible, context);
                            l = times_2(l, R - n);
                            R = n;
                            pass = 1;
                            continue;
                        }
                        l += sum;
                        store_weights(tm + weight_col<QP>(j * (kC / 16)), pk);
                        pass = 0;
                        ++j;
                    }
                    tmem_wait_st();
                    tc_before();
                }
                // this step's values and the next keys, there for long: waited for before the others are
                if (tid == 0 && ok) {
                    const bool next = s + 1 < n_steps;   // else the values' again
                    ok = mbar_spin(&sm.bars[kBarV], ph, &sm.bars[next ? kBarK : kBarV], next ? ph ^ 1u : ph, abort_flag, p.wait_limit);
                }
                __syncwarp();
                // every softmax warp comes here at every step, and all leave together
                ok = !worker_any<kSoft>(!ok);
                if (!ok) break;
                if (tid == 0) {
                    issue_context(s);
                    if (s + 1 < n_steps) issue_scores(s + 1);
                }
                __syncwarp();
            }
            // every product issued is done before the tile ends, after an abort too
            if (tid == 0) {
                umma_commit(&sm.bars[kBarDone]);
                int own = 0;
                mbar_wait(&sm.bars[kBarDone], tiles & 1u, &own);
                if (own) sm.abort = 1;
            }
            __syncwarp();
            // the last product's end
            if (ok && n_steps > 0) ok = mbar_wait(&sm.bars[kBarO], (it + n_steps - 1) & 1u, abort_flag, p.wait_limit);
            ok = __all_sync(kFull, ok);
            if (ok) {
                tc_after();
                const bool summed = n_steps > C::kFlush;
                if (summed) flush(false);
                const float4* tot = reinterpret_cast<const float4*>(p.ws_tot) + (int64_t)blockIdx.x * (D / 4) * kM + tid;
                const float sum = summed ? sm.sum_tot[tid] : l, ref = summed ? sm.ref_tot[tid] : R, inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                const bool live = tid < seg.vecs;
                QT* out = static_cast<QT*>(p.out) + (live ? gqa_vector<D>(p, seg, seg.vec0 + tid) : 0);
                float4* dst = reinterpret_cast<float4*>(p.ws_o) + (int64_t)max(seg.slot, 0) * (D / 4) * kM + tid;
#pragma unroll 1
                for (int k = 0; k < D / 32; ++k) {
                    uint32_t o[32];
                    if (n_steps > 0 && !summed) {
                        tmem_ld32(tm + C::kColO + 32 * k, o);
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float x[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = n_steps > 0 && !summed ? __uint_as_float(o[8 * i + e]) : 0.0f;
                        if (summed) {
                            const float4 a = tot[(8 * k + 2 * i) * kM], b = tot[(8 * k + 2 * i + 1) * kM];
                            x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
                            x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] *= inv;
                        if (seg.slot < 0) {
                            if (live) store8(out + 32 * k + 8 * i, x);
                        } else {
                            dst[(8 * k + 2 * i) * kM] = make_float4(x[0], x[1], x[2], x[3]);
                            dst[(8 * k + 2 * i + 1) * kM] = make_float4(x[4], x[5], x[6], x[7]);
                        }
                    }
                }
                if (seg.slot >= 0)
                    p.ws_ml[seg.slot * kM + tid] = make_float2(sum == 0.0f ? kNone : ref + log2f(sum), 0.0f);
                if (tid == 0 && seg.slot >= 0 && seg.u0 == 0)
                    p.cuts[blockIdx.x] = GqaCut{seg.count, seg.h, seg.vec0, seg.vecs, seg.q0};
            }
        } else {
            // ---- codes to f16: rows 32 (warp - 4) .. of each step ---------------------
            const int w0 = 32 * (warp - 4);
            const int32_t in_page = (1 << p.shift) - 1;
            // page of the warp's rows 0 .. 15 and 16 .. 31 of step s: lanes 0 and 1
            auto page_of = [&](int s) {
                const int32_t r = (u0 + s) * kN + w0 + 16 * (lane & 1);
                return s < n_steps && r < seg.limit ? gqa_page(p, seg.b, r) : -1;
            };
            auto rows_of = [&](int32_t page, int s, int64_t (&at)[2]) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const int32_t id = __shfl_sync(kFull, page, g);
                    at[g] = id < 0 ? -1 : (((int64_t)id * p.n_kv + seg.h) << p.shift) + (((u0 + s) * kN + w0 + 16 * g) & in_page);
                }
            };
            auto scale_of = [&](const int64_t (&at)[2]) {
                const int64_t x = lane < 16 ? at[0] : at[1];
                return x < 0 ? make_float2(0.0f, 0.0f) : p.scales[x + (lane & 15)];
            };
            // keys and values take turns in the same registers: the values of a step are needed a
            // softmax after its keys, the next keys a product later still
            Codes<D> codes;
            int64_t at[2];
            int32_t page = page_of(0);
            rows_of(page, 0, at);
            codes.load(p.k_codes, at, lane);
            float2 sc = scale_of(at);
            page = page_of(1);
            for (int s = 0; s < n_steps; ++s) {
                const uint32_t ph = (it + s) & 1u;
                bool ok = s == 0 || mbar_wait(&sm.bars[kBarS], ph ^ 1u, abort_flag, p.wait_limit);
                if (!__all_sync(kFull, ok)) break;
                codes.store(raw + C::kOffK + w0 * 128, lane);
                codes.load(p.v_codes, at, lane);
                if ((u0 + s) * kN + kN > all && codes.mend(lane)) sc.y = __uint_as_float(0x7fffffffu);
                sm.sk[ph][w0 + lane] = key_scale(sc.x);
                sm.sv[ph][w0 + lane] = sc.y;
                const float top = warp_max(fabsf(sc.y));
                if (lane == 0) sm.sv_top[ph][warp - 4] = top;
                fence_async_smem();
                mbar_arrive(&sm.bars[kBarK]);
                rows_of(page, s + 1, at);
                sc = scale_of(at);
                page = page_of(s + 2);
                ok = s == 0 || mbar_wait(&sm.bars[kBarO], ph ^ 1u, abort_flag, p.wait_limit);
                if (!__all_sync(kFull, ok)) break;
                codes.store(raw + C::kOffV + w0 * 128, lane);
                fence_async_smem();
                mbar_arrive(&sm.bars[kBarV]);
                codes.load(p.k_codes, at, lane);
            }
        }
        it += n_steps;
        tc_before();
        __syncthreads();
        tc_after();
        if (sm.abort || seg.last) break;
        __syncthreads();   // the segment is read
        if (warp == 4) {
            Walk walk = sm.walk;
            const bool more = walk.next(p);
            __syncwarp();
            if (lane == 0) {
                sm.walk = walk;
                sm.more = more && walk.get(p, sm.seg);
            }
        }
        __syncthreads();
        if (!sm.more) break;
    }
    tc_before();
    __syncthreads();
    if (tid == 0 && sm.abort) set_err(p.err, KVQ_ERR_TIMEOUT);
    if (warp == 4) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols));
}

// Cut tiles joined: CTA (c, k) the dims 16 k .. of the tile that CTA c began, a vector a thread in
// each of two groups that share the states.
constexpr int kMergeGroups = 2, kMergeDims = 16;
template <int D, typename QT>
__global__ void __launch_bounds__(kM * kMergeGroups) gqa_tc_merge_kernel(const __grid_constant__ GqaParams p) {
    constexpr int kE = kMergeDims / 4;
    __shared__ float2 stat[kMergeGroups][kM];
    __shared__ float4 part[kMergeGroups][kE][kM];
    grid_dependency_wait();
    launch_dependents();
    const int first = blockIdx.x, k = blockIdx.y, v = threadIdx.x % kM, grp = threadIdx.x / kM;
    const GqaCut cut = p.cuts[first];
    if (cut.count == 0) return;
    auto take = [](float4& o, const float4& x, float a, float b) {
        o.x = o.x * a + x.x * b;
        o.y = o.y * a + x.y * b;
        o.z = o.z * a + x.z * b;
        o.w = o.w * a + x.w * b;
    };
    float top = kNone, sum = 0.0f;
    float4 o[kE] = {};
#pragma unroll 4
    for (int i = grp; i < cut.count; i += kMergeGroups) {
        const int sl = Walk::slot(first + i, first);
        const float L = __ldcg(&p.ws_ml[sl * kM + v]).x;
        const float4* src = reinterpret_cast<const float4*>(p.ws_o) + ((int64_t)sl * (D / 4) + kE * k) * kM + v;
        float4 x[kE];
#pragma unroll
        for (int e = 0; e < kE; ++e) x[e] = __ldcg(src + e * kM);
        const float n = fmaxf(top, L), a = ex2(top - n), b = L == kNone ? 0.0f : ex2(L - n);
        sum = sum * a + b;
        top = n;
#pragma unroll
        for (int e = 0; e < kE; ++e) take(o[e], x[e], a, b);
    }
    stat[grp][v] = make_float2(top, sum);
#pragma unroll
    for (int e = 0; e < kE; ++e) part[grp][e][v] = o[e];
    __syncthreads();
    if (grp != 0 || v >= cut.vecs) return;
#pragma unroll
    for (int w = 1; w < kMergeGroups; ++w) {
        const float2 s = stat[w][v];
        const float n = fmaxf(top, s.x), a = ex2(top - n), b = ex2(s.x - n);
        sum = sum * a + s.y * b;
        top = n;
#pragma unroll
        for (int e = 0; e < kE; ++e) take(o[e], part[w][e][v], a, b);
    }
    GqaSegment seg;
    seg.h = cut.h;
    seg.q0 = cut.q0;
    QT* out = static_cast<QT*>(p.out) + gqa_vector<D>(p, seg, cut.vec0 + v) + kMergeDims * k;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int e = 0; e < kE; e += 2) {
        const float4 a = o[e], b = o[e + 1];
        const float x[8] = {a.x * inv, a.y * inv, a.z * inv, a.w * inv, b.x * inv, b.y * inv, b.z * inv, b.w * inv};
        store8(out + 4 * e, x);
    }
}

template <int D, int QP, typename QT>
cudaError_t launch_kernel(const GqaParams& p, cudaStream_t stream) {
    using C = Cfg<D, QP>;
    constexpr size_t smem = C::kOffMisc + sizeof(Misc);
    static_assert(smem <= 227 * 1024, "shared memory");
    constexpr int ctas = 152 * C::kCtas;
    cudaError_t e = cudaFuncSetAttribute(gqa_tc_kernel<D, QP, QT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    timing_mark(stream, 0);
    e = launch_chained(gqa_tc_kernel<D, QP, QT>, ctas, kNT, smem, stream, p);
    timing_mark(stream, 1);
    if (e == cudaSuccess) e = launch_chained(gqa_tc_merge_kernel<D, QT>, dim3(ctas, D / kMergeDims), kM * kMergeGroups, 0, stream, p);
    timing_mark(stream, 2);
    return e;
}

}  // namespace

// Partial states, two a CTA, and totals.
size_t gqa_tc_state_bytes(int32_t head_dim) {
    const size_t ctas = head_dim == 256 ? 152 : 304;
    return ctas * kM * (2 * (sizeof(float2) + head_dim * sizeof(float)) + head_dim * sizeof(float));
}
bool gqa_tc_supported(int32_t head_dim, kvq_dtype dt) { return head_dim != 256 || dt == KVQ_BF16; }

cudaError_t launch_gqa_tc(const GqaParams& p0, int32_t head_dim, kvq_dtype dt, void* state, cudaStream_t stream) {
    GqaParams p = p0;
    const size_t ctas = head_dim == 256 ? 152 : 304;
    p.ws_ml = static_cast<float2*>(state);
    p.ws_o = reinterpret_cast<float*>(p.ws_ml + 2 * ctas * kM);
    p.ws_tot = p.ws_o + 2 * ctas * kM * head_dim;
    p.stall_polls = test_stall_polls();
    p.wait_limit = p.stall_polls > 0 ? p.stall_polls : kWaitLimit;
    switch (head_dim) {
        case 64:
            return dt == KVQ_BF16 ? launch_kernel<64, 1, __nv_bfloat16>(p, stream) : launch_kernel<64, 2, float>(p, stream);
        case 128:
            return dt == KVQ_BF16 ? launch_kernel<128, 1, __nv_bfloat16>(p, stream) : launch_kernel<128, 2, float>(p, stream);
        default: return dt == KVQ_BF16 ? launch_kernel<256, 1, __nv_bfloat16>(p, stream) : cudaErrorInvalidValue;
    }
}

}  // namespace kvq
