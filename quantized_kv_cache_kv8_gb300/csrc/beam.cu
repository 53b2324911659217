// beam.cu -- beam search's selection: the best continuations of every request over
// its beams and the vocabulary, straight from the logits.
//
//   score(b, v) = cum_b + x_bv - lse_b,   lse_b = log sum_v exp(x_bv)
// and the `keep` best pairs (b, v) of a request, best first; ties go to the lower beam,
// within a beam to the larger logit, then to the lower token.
//
// What bounds it: reading the logits, once.  A beam's row is cut into slices, one CTA
// each.  A thread keeps 4 vectors of 16 bytes in flight and sums 2^((x - r) l) as it goes,
// l = log2(e) in f32 and r a reference of its own, in f32 (4 partial sums); from there on in f64.
// With the same l in the sum and behind it, the error of l moves a score by 1.3e-8 of
// the row's entropy, not of its logits.
//
// Selection without sorting.  The `keep`-th largest of the threads' maxima over the
// first trip is a bound that at least `keep` elements reach, so elements below it are
// out, and so are later ones that only equal it (their index is higher).  What passes goes to a
// list in shared memory, about `keep` elements a trip, and each finds its rank by
// counting.  Should the list overflow (ascending or equal logits), the slice's best are found
// one after another by maxima over the slice, `keep` passes in L2: slower, the same answer.
// The slice lists of a request are merged by the CTA that comes last, a head a lane.
#include "gqa.cuh"
#include "tc_common.cuh"

#include <algorithm>

namespace kvq {
namespace {

using tc::ex2;

constexpr int kNT = 256, kWarps = kNT / 32;
constexpr int kTrip = 4;             // vectors of a thread and trip
constexpr int kList = 1024;          // elements that may pass the bound
constexpr int kMaxKeep = 64, kMaxBeams = 32;
constexpr int kMaxLists = kNT;       // slice lists of a request
constexpr int kMaxCand = 2048;       // their elements
constexpr float kL = tc::kLog2e;

struct BeamParams {
    const void* logits;
    int64_t stride;       // elements between rows
    int64_t vocab;
    int32_t n_beams, keep, splits;
    int64_t per_split;    // vectors
    const float* scores;
    float* out_scores;
    int32_t* parents;
    int32_t* tokens;
    uint32_t* tickets;    // [n_seq]
    double2* sums;        // [rows][splits]: reference, sum
    int32_t* counts;      // [rows][splits]
    uint64_t* keys;       // [rows][splits][keep]
};

// Larger key: larger value, then lower index.  -0 and 0 are the same value.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint64_t make_key(float x, uint32_t index) {
    return ((uint64_t)ordered(x) << 32) | (uint32_t)~index;
}
__device__ __forceinline__ float key_value(uint64_t k) {
    const uint32_t o = (uint32_t)(k >> 32);
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint32_t key_index(uint64_t k) { return ~(uint32_t)k; }

// A row in vectors of 16 bytes, counted from its first element wherever that lies: beams
// of the same logits get the same sums, bit for bit.  NaN and what lies outside the row
// are -inf.
template <typename T>
struct Row {
    static constexpr int V = 16 / sizeof(T);
    const T* x;
    uint32_t shift;    // bytes between the 16-byte boundary before the row and it
    int64_t n;
    __device__ __forceinline__ Row(const T* p, int64_t vocab) : x(p), shift((uint32_t)((uintptr_t)p & 15u)), n(vocab) {}
    __device__ __forceinline__ int64_t vectors() const { return (n + V - 1) / V; }
    static __device__ __forceinline__ uint4 ldg(const char* p) {
        uint4 r;
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                     : "l"(p));
        return r;
    }
    __device__ __forceinline__ uint4 load(int64_t v) const {
        const int64_t e = v * V;
        const char* at = reinterpret_cast<const char*>(x + e);
        if (e + V <= n) {
            if (shift == 0) return ldg(at);
            // both aligned pieces hold elements of the vector
            const uint4 lo = *reinterpret_cast<const uint4*>(at - shift), hi = *reinterpret_cast<const uint4*>(at - shift + 16);
            uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            if (shift & 8) {
#pragma unroll
                for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
            }
            if (shift & 4) {
#pragma unroll
                for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
            }
            const uint32_t bits = 8 * (shift & 3);
            return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                              __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
        }
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                w[i] = e + i < n ? reinterpret_cast<const uint32_t*>(x)[e + i] : 0xff800000u;
            } else {
                const int64_t a = e + 2 * i;
                const uint32_t lo = a < n ? reinterpret_cast<const uint16_t*>(x)[a] : 0xff80u;
                const uint32_t hi = a + 1 < n ? reinterpret_cast<const uint16_t*>(x)[a + 1] : 0xff80u;
                w[i] = lo | (hi << 16);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ static __forceinline__ void floats(uint4 r, float (&f)[V]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = fmaxf(__uint_as_float(w[i]), -INFINITY);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 none = __halves2bfloat162(__ushort_as_bfloat16(0xff80), __ushort_as_bfloat16(0xff80));
                const __nv_bfloat162 v = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), none);
                const uint32_t u = *reinterpret_cast<const uint32_t*>(&v);
                f[2 * i] = __uint_as_float(u << 16);
                f[2 * i + 1] = __uint_as_float(u & 0xffff0000u);
            }
        }
    }
};

// sum e^(x - ref) of some elements; two of them joined (nothing so far: -inf, 0).
struct Mass {
    double ref, sum;
};
__device__ __forceinline__ Mass join(Mass a, Mass b) {
    const double t = fmax(a.ref, b.ref);
    return Mass{t, (a.ref == t ? a.sum : a.sum * (double)ex2((float)(a.ref - t) * kL)) +
                       (b.ref == t ? b.sum : b.sum * (double)ex2((float)(b.ref - t) * kL))};
}

struct Shared {
    union {
        uint64_t list[kList];
        uint64_t cand[kMaxCand];
    };
    float maxima[kNT];
    Mass warp_mass[kWarps];
    uint64_t warp_key[kWarps];
    double lse[kMaxBeams];
    float cum[kMaxBeams], top[kMaxBeams];
    int32_t count[kMaxLists];
    uint64_t best_key[kWarps][kMaxKeep];
    uint64_t best_score[kWarps][kMaxKeep];
    uint8_t best_beam[kWarps][kMaxKeep];
    int32_t best_count[kWarps];
    int n_list, last;
};

__device__ __forceinline__ uint64_t ordered64(double x) {
    const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
    return b ^ ((b >> 63) ? ~0ull : 0x8000000000000000ull);
}
__device__ __forceinline__ double from_ordered64(uint64_t o) {
    return __longlong_as_double((long long)(o ^ ((o >> 63) ? 0x8000000000000000ull : ~0ull)));
}
// The lane among `who` with the largest v (uniform); those that share it.
__device__ __forceinline__ unsigned warp_best(unsigned who, uint64_t v, int lane) {
    const bool in = (who >> lane) & 1u;
    const uint32_t hi = __reduce_max_sync(kFull, in ? (uint32_t)(v >> 32) : 0u);
    who = __ballot_sync(kFull, in && (uint32_t)(v >> 32) == hi);
    if ((who & (who - 1)) == 0u) return who;
    const bool in2 = (who >> lane) & 1u;
    const uint32_t lo = __reduce_max_sync(kFull, in2 ? (uint32_t)v : 0u);
    return __ballot_sync(kFull, in2 && (uint32_t)v == lo);
}

// `keep` best of sorted lists, one a lane: score(i) the ordered score of element i of the
// lane's list (0: none), key(i) its key.  take(k, lane, i) is called by the lane that holds the k-th.
template <class Score, class Key, class Take>
__device__ __forceinline__ int merge_lists(int keep, int n, int beam, int lane, Score score, Key key, Take take) {
    int i = 0;
    uint64_t s = n > 0 ? score(0) : 0ull;
    uint64_t k = s ? key(0) : 0ull;
    int found = 0;
    for (; found < keep; ++found) {
        unsigned who = __ballot_sync(kFull, s != 0ull);
        if (who == 0u) break;
        who = warp_best(who, s, lane);
        if (who & (who - 1)) {   // the same score: the lower beam, then the better key
            const uint32_t b = __reduce_min_sync(kFull, (who >> lane) & 1u ? (uint32_t)beam : 0xffffffffu);
            who = __ballot_sync(kFull, ((who >> lane) & 1u) && (uint32_t)beam == b);
            if (who & (who - 1)) who = warp_best(who, k, lane);
        }
        if (lane == __ffs(who) - 1) {
            take(found, i, s, k);
            ++i;
            s = i < n ? score(i) : 0ull;
            k = s ? key(i) : 0ull;
        }
    }
    return found;
}

template <typename T>
__global__ void __launch_bounds__(kNT) beam_select_kernel(const __grid_constant__ BeamParams p) {
    using R = Row<T>;
    constexpr int V = R::V;
    __shared__ Shared sm;
    launch_dependents();
    grid_dependency_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / p.splits;
    const int split = (int)(blockIdx.x - row * p.splits);
    const R x(static_cast<const T*>(p.logits) + row * p.stride, p.vocab);
    const int64_t v0 = split * p.per_split, v1 = min(v0 + p.per_split, x.vectors());
    const int keep = p.keep;
    if (tid == 0) sm.n_list = 0;

    float ref = -INFINITY;
    float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    float bound = -INFINITY;
    bool first = true;
    for (int64_t t0 = v0; t0 < v1; t0 += kTrip * kNT) {
        uint4 r[kTrip];
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < kTrip; ++u) {
            const int64_t v = t0 + u * kNT + tid;
            r[u] = v < v1 ? x.load(v)
                          : (sizeof(T) == 4 ? make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u)
                                            : make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u));
        }
#pragma unroll
        for (int u = 0; u < kTrip; ++u) {
            float f[V];
            R::floats(r[u], f);
#pragma unroll
            for (int i = 0; i < V; ++i) top = fmaxf(top, f[i]);
        }
        if (top > -INFINITY) {
            if (top == INFINITY || ref == INFINITY) {   // infinite logits share the whole mass
                if (ref != INFINITY) s4[0] = s4[1] = s4[2] = s4[3] = 0.0f;
                ref = INFINITY;
#pragma unroll
                for (int u = 0; u < kTrip; ++u) {
                    float f[V];
                    R::floats(r[u], f);
#pragma unroll
                    for (int i = 0; i < V; ++i) s4[i & 3] += f[i] == INFINITY ? 1.0f : 0.0f;
                }
            } else {
                if (top > ref + 16.0f) {   // sums of terms up to e^16 stay well inside f32
                    const float k = ref == -INFINITY ? 0.0f : ex2((ref - top) * kL);
#pragma unroll
                    for (int i = 0; i < 4; ++i) s4[i] *= k;
                    ref = top;
                }
#pragma unroll
                for (int u = 0; u < kTrip; ++u) {
                    float f[V];
                    R::floats(r[u], f);
#pragma unroll
                    for (int i = 0; i < V; ++i) s4[i & 3] += ex2((f[i] - ref) * kL);
                }
            }
        }
        if (first) {
            sm.maxima[tid] = top;
            __syncthreads();
            // rank of this thread's maximum; the one of rank keep - 1 is the bound
            int rank = 0;
            for (int i = 0; i < kNT; i += 4) {
                const float4 o = *reinterpret_cast<const float4*>(&sm.maxima[i]);
                rank += o.x > top || (o.x == top && i < tid);
                rank += o.y > top || (o.y == top && i + 1 < tid);
                rank += o.z > top || (o.z == top && i + 2 < tid);
                rank += o.w > top || (o.w == top && i + 3 < tid);
            }
            __syncthreads();
            if (rank == keep - 1) sm.maxima[0] = top;
            __syncthreads();
            bound = sm.maxima[0];
        }
        if (top > bound || (first && top == bound && top > -INFINITY)) {
#pragma unroll
            for (int u = 0; u < kTrip; ++u) {
                float f[V];
                R::floats(r[u], f);
                const int64_t e = (t0 + u * kNT + tid) * V;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (f[i] > bound || (first && f[i] == bound && f[i] > -INFINITY)) {
                        const int at = atomicAdd(&sm.n_list, 1);
                        if (at < kList) sm.list[at] = make_key(f[i], (uint32_t)(e + i));
                    }
            }
        }
        first = false;
    }
    // the slice's sum: references and partial sums joined in f64, in a fixed order
    Mass mass{ref, ((double)s4[0] + s4[1]) + ((double)s4[2] + s4[3])};
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        mass = join(mass, Mass{__shfl_xor_sync(kFull, mass.ref, o), __shfl_xor_sync(kFull, mass.sum, o)});
    if (lane == 0) sm.warp_mass[warp] = mass;
    __syncthreads();
    const int n = sm.n_list;
    const int64_t out = row * p.splits + split;
    if (tid == 0) {
        mass = sm.warp_mass[0];
        for (int w = 1; w < kWarps; ++w) mass = join(mass, sm.warp_mass[w]);
        p.sums[out] = make_double2(mass.ref, mass.sum);
    }
    uint64_t* keys = p.keys + out * keep;
    if (n <= kList) {
        for (int i = tid; i < n; i += kNT) {
            const uint64_t k = sm.list[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += sm.list[j] > k;
            if (rank < keep) keys[rank] = k;
        }
        if (tid == 0) p.counts[out] = min(n, keep);
    } else {
        uint64_t before = ~0ull;   // the key found last
        int found = 0;
        for (; found < keep; ++found) {
            uint64_t best = 0ull;
            for (int64_t v = v0 + tid; v < v1; v += kNT) {
                float f[V];
                R::floats(x.load(v), f);
                const int64_t e = v * V;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (f[i] > -INFINITY) {
                        const uint64_t k = make_key(f[i], (uint32_t)(e + i));
                        if (k < before && k > best) best = k;
                    }
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) best = max(best, __shfl_xor_sync(kFull, best, o));
            __syncthreads();
            if (lane == 0) sm.warp_key[warp] = best;
            __syncthreads();
            for (int w = 0; w < kWarps; ++w) best = max(best, sm.warp_key[w]);
            if (best == 0ull) break;
            if (tid == 0) keys[found] = best;
            before = best;
        }
        if (tid == 0) p.counts[out] = found;
    }

    // the request's last CTA merges the slices
    const int64_t seq = row / p.n_beams;
    const int lists = p.n_beams * p.splits;
    __threadfence();
    __syncthreads();
    if (tid == 0) sm.last = atomicAdd(p.tickets + seq, 1u) == (uint32_t)(lists - 1);
    __syncthreads();
    if (!sm.last) return;
    __threadfence();
    if (tid == 0) p.tickets[seq] = 0u;
    const int64_t list0 = seq * lists;
    for (int i = tid; i < lists * keep; i += kNT) sm.cand[i] = __ldcg(p.keys + list0 * keep + i);
    if (tid < lists) sm.count[tid] = __ldcg(p.counts + list0 + tid);
    if (tid < p.n_beams) {
        Mass mass{-INFINITY, 0.0};
        float top = -INFINITY;
        for (int i = 0; i < p.splits; ++i) {
            const int64_t l = list0 + tid * p.splits + i;
            const double2 o = __ldcg(p.sums + l);
            mass = join(mass, Mass{o.x, o.y});
            if (__ldcg(p.counts + l) > 0) top = fmaxf(top, key_value(__ldcg(p.keys + l * keep)));
        }
        // log of the mass against the largest logit
        sm.top[tid] = top;
        sm.lse[tid] = top == INFINITY ? log(mass.sum) : (mass.ref - (double)top) + log2(mass.sum) / (double)kL;
        sm.cum[tid] = p.scores[seq * p.n_beams + tid];
    }
    __syncthreads();
    const int beam = tid < lists ? tid / p.splits : 0;
    const float cum = sm.cum[beam];
    const float top = sm.top[beam];
    const bool alive = fabsf(cum) <= 3.402823466e38f;
    const double lse = sm.lse[beam];
    const uint64_t* mine = sm.cand + tid * keep;
    auto score = [&](int i) -> uint64_t {
        const float v = key_value(mine[i]);
        const double sc = (double)cum + ((v == top ? 0.0 : (double)v - (double)top) - lse);
        return sc > -INFINITY ? ordered64(sc) : 0ull;   // beside an infinite logit
    };
    const int n_mine = tid < lists && alive ? sm.count[tid] : 0;
    const int warps = (lists + 31) / 32;
    float* os = p.out_scores + seq * keep;
    int32_t* op = p.parents + seq * keep;
    int32_t* ot = p.tokens + seq * keep;
    auto emit = [&](int k, uint64_t sc, uint64_t key, int bm) {
        os[k] = (float)from_ordered64(sc);
        op[k] = (int32_t)(seq * p.n_beams + bm);
        ot[k] = (int32_t)key_index(key);
    };
    int found = 0;
    if (warps == 1) {
        if (warp == 0)
            found = merge_lists(keep, n_mine, beam, lane, score, [&](int i) { return mine[i]; },
                                [&](int k, int, uint64_t sc, uint64_t key) { emit(k, sc, key, beam); });
    } else {
        if (warp < warps) {
            const int f = merge_lists(keep, n_mine, beam, lane, score, [&](int i) { return mine[i]; },
                                      [&](int k, int, uint64_t sc, uint64_t key) {
                                          sm.best_score[warp][k] = sc;
                                          sm.best_key[warp][k] = key;
                                          sm.best_beam[warp][k] = (uint8_t)beam;
                                      });
            if (lane == 0) sm.best_count[warp] = f;
        }
        __syncthreads();
        if (warp == 0) {
            // lists of several beams: a head's beam is its element's
            const int l = min(lane, kWarps - 1), nl = lane < warps ? sm.best_count[l] : 0;
            int i = 0;
            uint64_t s_ = nl > 0 ? sm.best_score[l][0] : 0ull;
            for (; found < keep; ++found) {
                unsigned who = __ballot_sync(kFull, s_ != 0ull);
                if (who == 0u) break;
                who = warp_best(who, s_, lane);
                if (who & (who - 1)) {
                    const bool in = (who >> lane) & 1u;
                    const uint32_t bm = in ? sm.best_beam[l][i] : 0xffffffffu;
                    const uint32_t b = __reduce_min_sync(kFull, bm);
                    who = __ballot_sync(kFull, in && bm == b);
                    if (who & (who - 1)) who = warp_best(who, (who >> lane) & 1u ? sm.best_key[l][i] : 0ull, lane);
                }
                if (lane == __ffs(who) - 1) {
                    emit(found, s_, sm.best_key[l][i], sm.best_beam[l][i]);
                    ++i;
                    s_ = i < nl ? sm.best_score[l][i] : 0ull;
                }
            }
        }
    }
    if (warp == 0)
        for (int k = found + lane; k < keep; k += 32) {   // fewer continuations than asked for
            os[k] = -INFINITY;
            op[k] = -1;
            ot[k] = -1;
        }
}

// Slices of a row: CTAs for 8 a SM, slices of at least 16 KB, lists within a request's limits.
int splits_for(int64_t rows, int32_t n_beams, int64_t vocab, int32_t keep, int size) {
    int64_t s = (152 * 8 + rows - 1) / std::max<int64_t>(1, rows);
    s = std::min<int64_t>(s, vocab * size / 16384);
    s = std::min<int64_t>(s, std::min(kMaxLists / n_beams, kMaxCand / (n_beams * keep)));
    return (int)std::max<int64_t>(1, s);
}
size_t round_up(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

// Sized for the slices of either type (f32 rows have the most).
size_t beam_workspace_bytes(int32_t n_seq, int32_t n_beams, int64_t vocab, int32_t keep) {
    const int64_t rows = (int64_t)n_seq * n_beams;
    const size_t lists = (size_t)rows * splits_for(rows, n_beams, vocab, keep, 4);
    return kWsHeader + round_up((size_t)n_seq * 4) + lists * (sizeof(double2) + 8 * (size_t)keep + 4);
}

cudaError_t launch_beam_select(const void* logits, kvq_dtype dt, int64_t row_stride, int32_t n_seq, int32_t n_beams,
                               int64_t vocab, const float* scores, int32_t keep, float* out_scores, int32_t* parents,
                               int32_t* tokens, void* workspace, cudaStream_t stream) {
    BeamParams p{};
    const int64_t rows = (int64_t)n_seq * n_beams;
    const int size = dt == KVQ_BF16 ? 2 : 4;
    p.logits = logits;
    p.stride = row_stride;
    p.vocab = vocab;
    p.n_beams = n_beams;
    p.keep = keep;
    p.splits = splits_for(rows, n_beams, vocab, keep, size);
    const int64_t v = 16 / size, vectors = (vocab + v - 1) / v;
    p.per_split = (vectors + p.splits - 1) / p.splits;
    p.scores = scores;
    p.out_scores = out_scores;
    p.parents = parents;
    p.tokens = tokens;
    char* ws = static_cast<char*>(workspace) + kWsHeader;
    p.tickets = reinterpret_cast<uint32_t*>(ws);
    ws += round_up((size_t)n_seq * 4);
    p.sums = reinterpret_cast<double2*>(ws);
    p.keys = reinterpret_cast<uint64_t*>(p.sums + rows * p.splits);
    p.counts = reinterpret_cast<int32_t*>(p.keys + rows * p.splits * keep);
    const int64_t grid = rows * p.splits;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    return dt == KVQ_BF16 ? launch_chained(beam_select_kernel<__nv_bfloat16>, (unsigned)grid, kNT, 0, stream, p)
                          : launch_chained(beam_select_kernel<float>, (unsigned)grid, kNT, 0, stream, p);
}

}  // namespace kvq
