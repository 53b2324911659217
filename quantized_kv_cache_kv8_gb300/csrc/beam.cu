// beam.cu -- beam search's selection: the best continuations of every request over
// its beams and the vocabulary, straight from the logits.
//
//   score(b, v) = cum_b + x_bv - lse_b,   lse_b = log sum_v exp(x_bv)
// and the `keep` best pairs (b, v) of a request, best first; ties go to the lower beam,
// within a beam to the larger logit, then to the lower token.
//
// What bounds it: reading the logits, once.  A beam's row is cut into slices, one CTA
// each.  A thread asks for the next 4 vectors of 16 bytes and sums 2^(x l - r l) over the last 4,
// l = log2(e) in f32 and r a reference of its own, in f32, trip by trip; what the rounding of
// r l adds is a factor of the trip's sum.
// With the same l in the sum and behind it, the error of l moves a score by 1.3e-8 of
// the row's entropy, not of its logits.
//
// Selection without sorting.  Over the first trip each warp finds the (keep / 8)-th largest
// of its lanes' maxima; the least of these is a bound that at least `keep` elements reach, so
// elements below it are out, and later ones that only equal it too (their index is higher).  Vectors that hold
// more go to a list in shared memory; when it has grown by 16 their elements find their ranks by
// counting, the best `keep` stay and the last of them is the new bound.  Should a list overflow, the slice's
// best are found one after another by maxima over the slice, `keep` passes in L2: slower, the same answer.
// That takes ascending logits, or many equal to the bound (a mask of the type's lowest value instead of -inf:
// 64 requests of 8 beams over 131072 in bf16, 16 kept, 0.1% unmasked, 1.2 ms; 8 of 4 over 32768 in f32, 8 kept,
// 54 us), or a slice of more elements than the list holds in which some warp has fewer than keep / 8 lanes
// with any, so that there is no bound: rows of some 500 to 1900 in bf16, 500 to 900 in f32 (4 of 4 over 1000
// in bf16, 16 kept, 24 us, 64 kept 80).
// The slice lists of a request are merged by the CTA that comes last: their elements' scores, those
// out that the best full list's last beats, ranks among the rest.
//
// Measured: 64 requests of 8 beams over 131072 in bf16, 16 kept: 47 us, 2.8 TB/s.  A trip takes
// 1.4 us once all run, which is the memory's rate; the first, the list's first ranking in the third,
// and the end (ranks, the last CTA's merge) 4 us each.  8 of 4 over 32768 in f32, 8 kept: 11.4 us,
// the merge 4 of them.
#include "gqa.cuh"
#include "tc_common.cuh"

#include <algorithm>

namespace kvq {
namespace {

using tc::ex2;

constexpr int kNT = 256, kWarps = kNT / 32;
constexpr int kTrip = 4;             // vectors of a thread and trip (odd_sum lists them)
constexpr int kVec = 256;            // vectors that may hold elements past the bound
constexpr int kList = 512;           // such elements
constexpr int kMaxKeep = 64, kMaxBeams = 32;
constexpr int kMaxLists = kNT;       // slice lists of a request
constexpr int kMaxCand = 2048;       // their elements
constexpr float kL = tc::kLog2e;
constexpr float kMaxF = 3.402823466e38f;   // f32's largest

struct BeamParams {
    const void* logits;
    int64_t stride;       // elements between rows
    int64_t vocab;
    int32_t n_beams, keep, splits;
    uint32_t per_split;   // vectors
    const float* scores;
    float* out_scores;
    int32_t* parents;
    int32_t* tokens;
    uint32_t* tickets;    // [n_seq]
    float2* sums;         // [rows][splits]: reference, sum
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
__device__ __forceinline__ float from_ordered(uint32_t o) {
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ float key_value(uint64_t k) { return from_ordered((uint32_t)(k >> 32)); }
__device__ __forceinline__ uint32_t key_index(uint64_t k) { return ~(uint32_t)k; }

// A row in vectors of 16 bytes, counted from its first element wherever that lies: beams
// of the same logits get the same sums, bit for bit.  NaN and what lies outside the row
// are -inf.
template <typename T>
struct Row {
    static constexpr int V = 16 / sizeof(T);
    const char* x;
    uint32_t shift;    // bytes between the 16-byte boundary before the row and it
    uint32_t n, whole; // elements; whole vectors
    __device__ __forceinline__ Row(const T* p, int64_t vocab)
        : x(reinterpret_cast<const char*>(p)), shift((uint32_t)((uintptr_t)p & 15u)), n((uint32_t)vocab), whole(n / V) {}
    __device__ __forceinline__ uint32_t vectors() const { return (n + V - 1) / V; }
    // The vectors from, from + step, ...: `none` from `end` on.
    template <int N>
    __device__ __forceinline__ void load(uint4 (&r)[N], uint32_t from, uint32_t step, uint32_t end) const {
        if (shift == 0 && from + (N - 1) * step < min(end, whole)) {
            const char* at = x + (uint64_t)from * 16u;
#pragma unroll
            for (int u = 0; u < N; ++u) r[u] = ldg16(at + u * step * 16u);
        } else {
#pragma unroll
            for (int u = 0; u < N; ++u) r[u] = from + u * step < end ? load(from + u * step) : none();
        }
    }
    __device__ __noinline__ uint4 load(uint32_t v) const {
        const char* at = x + (uint64_t)v * 16u;
        if (v < whole) {
            if (shift == 0) return ldg16(at);
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
                w[i] = v * V + i < n ? reinterpret_cast<const uint32_t*>(at)[i] : 0xff800000u;
            } else {
                const uint32_t a = v * V + 2 * i;
                const uint32_t lo = a < n ? reinterpret_cast<const uint16_t*>(at)[2 * i] : 0xff80u;
                const uint32_t hi = a + 1 < n ? reinterpret_cast<const uint16_t*>(at)[2 * i + 1] : 0xff80u;
                w[i] = lo | (hi << 16);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // Nothing: -inf in every place.
    static __device__ __forceinline__ uint4 none() {
        const uint32_t w = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
        return make_uint4(w, w, w, w);
    }
    static __device__ __forceinline__ void floats(uint4 r, float (&f)[V]) {   // NaN as it is
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                f[i] = __uint_as_float(w[i]);
            } else {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
    static __device__ __forceinline__ float top(uint4 r) {   // NaN passed over
        if constexpr (sizeof(T) == 4) {
            return fmaxf(fmaxf(fmaxf(__uint_as_float(r.x), -INFINITY), __uint_as_float(r.y)),
                         fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
        } else {
            const auto v = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
            const __nv_bfloat162 m = __hmax2(__hmax2(v(r.x), v(r.y)), __hmax2(v(r.z), v(r.w)));
            const uint32_t u = *reinterpret_cast<const uint32_t*>(&m);
            return fmaxf(fmaxf(__uint_as_float(u << 16), -INFINITY), __uint_as_float(u & 0xffff0000u));
        }
    }
};

// sum e^(x - ref) of some elements; two of them joined (nothing so far: -inf, 0).
struct Mass {
    float ref, sum;
};
__device__ __forceinline__ Mass join(Mass a, Mass b) {
    const float t = fmaxf(a.ref, b.ref);
    return Mass{t, (a.ref == t ? a.sum : a.sum * ex2((a.ref - t) * kL)) + (b.ref == t ? b.sum : b.sum * ex2((b.ref - t) * kL))};
}

// A sum of two f32, |lo| at most half a unit of hi: 48 bits (f64 arithmetic is slow here, and
// every step of the merge would wait for it).
struct Wide {
    float hi, lo;
};
__device__ __forceinline__ Wide two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return Wide{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Wide add(Wide a, Wide b) {
    const Wide s = two_sum(a.hi, b.hi);
    return two_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
// log s = k ln 2 + log m, m in [1, 2): logf's error is 2^-24 of log 2, k ln 2 is exact to 2^-48.
__device__ __forceinline__ Wide wide_log(float s) {
    const int k = (int)(__float_as_uint(s) >> 23) - 127;
    const float m = __uint_as_float((__float_as_uint(s) & 0x007fffffu) | 0x3f800000u);
    const float hi = 0.693147182464599609375f, lo = -1.904654299957768e-9f, f = (float)k;   // ln 2 in two
    const float p = __fmul_rn(f, hi);
    return add(Wide{p, __fadd_rn(__fmaf_rn(f, hi, -p), __fmul_rn(f, lo))}, Wide{logf(m), 0.0f});
}

struct Shared {
    union alignas(16) {
        uint64_t list[kList + 2];   // read in pairs
        uint64_t cand[kMaxCand];
    };
    Mass warp_mass[kWarps];
    uint64_t warp_key[kWarps];
    float warp_bound[kWarps];
    Wide base[kMaxBeams];    // cum - log of the mass against the largest logit
    float cum[kMaxBeams], top[kMaxBeams];
    int32_t count[kMaxLists];
    float2 mass[kMaxLists];
    uint64_t floor;
    int n_best, warp_count[kWarps];
    alignas(16) uint64_t best[kMaxCand + 2];
    uint16_t best_at[kMaxCand];
    uint4 vec[kVec];
    uint32_t vec_id[kVec];
    int n_vec, n_list, last;
};

__device__ __forceinline__ uint64_t ordered64(Wide x) { return ((uint64_t)ordered(x.hi) << 32) | ordered(x.lo); }
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
// take(i, rank) for each of the first n keys: rank, how many are larger or, being equal, before(j, i)
// (a list of one slice has no equal keys: they hold the token).
// By the whole CTA; as many threads share a key as there are for one.
template <bool EQUALS, class Before, class Take>
__device__ __forceinline__ void rank_all(const uint64_t* list, int n, Before before, Take take) {
    int share = 1;
    while (share < 8 && 2 * share * n <= kNT) share *= 2;
    const int part = threadIdx.x & (share - 1);
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += kNT / share) {
        const int i = i0 + (int)threadIdx.x / share;
        const uint64_t k = i < n ? list[i] : ~0ull;
        int rank = 0, same = 0;
#pragma unroll 4
        for (int j = 2 * part; j < n; j += 2 * share) {
            const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(list + j);
            rank += x.x > k;
            rank += j + 1 < n && x.y > k;
            if (EQUALS) same += (x.x == k) + (j + 1 < n && x.y == k);
        }
        for (int o = 1; o < share; o <<= 1) {
            rank += __shfl_xor_sync(kFull, rank, o);
            if (EQUALS) same += __shfl_xor_sync(kFull, same, o);
        }
        if (part != 0 || i >= n) continue;
        if constexpr (EQUALS)
            if (same > 1) {
#pragma unroll 1
                for (int j = 0; j < n; ++j) rank += list[j] == k && j != i && before(j, i);
            }
        take(i, rank);
    }
}
// Elements of the listed vectors that reach the bound, to the list of keys.  By the whole CTA; the
// vectors are stored, the keys need a barrier.
template <typename T>
__device__ __forceinline__ void expand(Shared& sm, int n_vec, float bound) {
    constexpr int V = Row<T>::V;
    for (int i = threadIdx.x; i < n_vec * V; i += kNT) {
        const int at = i / V, e = i % V;
        const float f = sizeof(T) == 4 ? reinterpret_cast<const float*>(&sm.vec[at])[e]
                                       : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(&sm.vec[at])[e] << 16);
        if (f >= bound && f > -INFINITY) {
            const int to = atomicAdd(&sm.n_list, 1);
            if (to < kList) sm.list[to] = make_key(f, sm.vec_id[at] * V + e);
        }
    }
}
// The sum of a trip that holds NaN, infinite logits (these share the whole mass: their number) or large ones.
template <typename T>
__device__ __noinline__ float odd_sum(const uint4 (&r)[kTrip], float ref) {
    constexpr int V = Row<T>::V;
    float s = 0.0f;
#pragma unroll 1
    for (int u = 0; u < kTrip; ++u) {
        float f[V];
        Row<T>::floats(u == 0 ? r[0] : u == 1 ? r[1] : u == 2 ? r[2] : r[3], f);
#pragma unroll
        for (int i = 0; i < V; ++i)
            s += f[i] == ref ? 1.0f : f[i] < ref ? ex2((f[i] - ref) * kL) : f[i] > ref ? ex2((f[i] - ref) * kL) : 0.0f;
    }
    return s;
}

template <typename T>
__global__ void __launch_bounds__(kNT, 4) beam_select_kernel(const __grid_constant__ BeamParams p) {
    using R = Row<T>;
    constexpr int V = R::V;
    __shared__ Shared sm;
    launch_dependents();
    grid_dependency_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / p.splits;
    const int split = (int)(blockIdx.x - row * p.splits);
    const R x(static_cast<const T*>(p.logits) + row * p.stride, p.vocab);
    const uint32_t v0 = min(split * p.per_split, x.vectors()), v1 = min(v0 + p.per_split, x.vectors());
    const int keep = p.keep, share = (keep + kWarps - 1) / kWarps;
    if (tid == 0) sm.n_list = sm.n_vec = 0;

    float ref = -INFINITY, sum = 0.0f;
    float bound = -INFINITY;
    bool first = true;
    uint4 even[kTrip], odd[kTrip];
    x.load(even, v0 + tid, kNT, v1);
    float rl = 0.0f, off = 1.0f;   // ref l in f32; 2^(what that rounding added)
    int trip = 0;
    const auto take = [&](uint32_t t0, const uint4 (&r)[kTrip]) {
        float vtop[kTrip], top = -INFINITY;
#pragma unroll
        for (int u = 0; u < kTrip; ++u) {
            vtop[u] = R::top(r[u]);
            top = fmaxf(top, vtop[u]);
        }
        if (top > -INFINITY) {
            if (top > ref + 16.0f || top == INFINITY) {   // sums of terms up to e^16 stay well inside f32
                sum = ref == top ? sum : ref == -INFINITY ? 0.0f : sum * ex2((ref - top) * kL);
                ref = top;
                rl = ref * kL;
                off = ex2(__fmaf_rn(-ref, kL, rl));
            }
            // two elements an instruction
            const uint64_t l2 = pack2(kL, kL), rl2 = pack2(-rl, -rl);
            uint64_t part[2] = {0ull, 0ull};
#pragma unroll
            for (int u = 0; u < kTrip; ++u) {
                float f[V];
                R::floats(r[u], f);
#pragma unroll
                for (int i = 0; i < V; i += 2) {
                    uint64_t t;
                    float a, b;
                    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(t) : "l"(pack2(f[i], f[i + 1])), "l"(l2), "l"(rl2));
                    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(t));
                    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(part[i / 2 & 1]) : "l"(part[i / 2 & 1]), "l"(pack2(ex2(a), ex2(b))));
                }
            }
            float a0, a1, b0, b1;
            asm("mov.b64 {%0, %1}, %2;" : "=f"(a0), "=f"(a1) : "l"(part[0]));
            asm("mov.b64 {%0, %1}, %2;" : "=f"(b0), "=f"(b1) : "l"(part[1]));
            const float all = ((a0 + a1) + (b0 + b1)) * off;
            // NaN or infinite logits, and such that ref l is off by more than 2^-4
            sum += all == all && fabsf(ref) <= 0x1p19f ? all : odd_sum<T>(r, ref);
        }
        if (first) {
            // a warp's share-th largest of its lanes' maxima; the least of the warps' is reached by
            // `keep` elements at least
            float mine = top, reach = -INFINITY;
            for (int k = 0; k < share; ++k) {
                const uint32_t best = __reduce_max_sync(kFull, ordered(mine));
                reach = from_ordered(best);
                const unsigned who = __ballot_sync(kFull, ordered(mine) == best);
                if (lane == __ffs(who) - 1) mine = -INFINITY;
            }
            if (lane == 0) sm.warp_bound[warp] = reach;
            __syncthreads();
            bound = sm.warp_bound[0];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) bound = fminf(bound, sm.warp_bound[w]);
        }
        if (top >= bound && top > -INFINITY) {
#pragma unroll
            for (int u = 0; u < kTrip; ++u)
                if (vtop[u] > bound || (first && vtop[u] == bound)) {
                    const int at = atomicAdd(&sm.n_vec, 1);
                    if (at < kVec) {
                        sm.vec[at] = r[u];
                        sm.vec_id[at] = t0 + u * kNT + tid;
                    }
                }
        }
        // once some more than `keep` are listed, the best `keep` stay and the last of them is the bound
        if (t0 + kTrip * kNT < v1 && (trip == 0 || trip == 2 || (trip & 15) == 15)) {
            __syncthreads();
            const int n_vec = sm.n_vec, listed = sm.n_list;
            __syncthreads();   // read by all before it grows
            if (n_vec + listed >= keep + 16 && n_vec <= kVec && listed <= kList) {
                expand<T>(sm, n_vec, bound);
                __syncthreads();
                const int n = sm.n_list;
                if (n <= kNT) {   // else the list waits
                    uint64_t k = 0ull;
                    int place = keep;
                    rank_all<false>(sm.list, n, 0, [&](int i, int rank) {
                        k = sm.list[i];
                        place = rank;
                    });
                    __syncthreads();
                    if (place < keep) sm.list[place] = k;
                    if (tid == 0) sm.n_list = min(n, keep);
                }
                if (tid == 0) sm.n_vec = 0;
                __syncthreads();
                if (n <= kNT && n >= keep) bound = key_value(sm.list[keep - 1]);
            }
        }
        first = false;
        ++trip;
    };
    constexpr uint32_t kSpan = kTrip * kNT;
#pragma unroll 1
    for (uint32_t t0 = v0; t0 < v1; t0 += 2 * kSpan) {
        x.load(odd, t0 + kSpan + tid, kNT, v1);
        take(t0, even);
        if (t0 + kSpan >= v1) break;
        x.load(even, t0 + 2 * kSpan + tid, kNT, v1);
        take(t0 + kSpan, odd);
    }
    // the slice's sum, joined in a fixed order
    Mass mass{ref, sum};
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        mass = join(mass, Mass{__shfl_xor_sync(kFull, mass.ref, o), __shfl_xor_sync(kFull, mass.sum, o)});
    if (lane == 0) sm.warp_mass[warp] = mass;
    __syncthreads();
    const int n_vec = sm.n_vec, listed = sm.n_list;
    __syncthreads();
    if (n_vec <= kVec && listed <= kList) expand<T>(sm, n_vec, bound);
    __syncthreads();
    const int n = n_vec <= kVec ? sm.n_list : kList + 1;
    const int64_t out = row * p.splits + split;
    if (tid == 0) {
        mass = sm.warp_mass[0];
        for (int w = 1; w < kWarps; ++w) mass = join(mass, sm.warp_mass[w]);
        p.sums[out] = make_float2(mass.ref, mass.sum);
    }
    uint64_t* keys = p.keys + out * keep;
    if (n <= kList) {
        rank_all<false>(sm.list, n, 0, [&](int i, int rank) {
            if (rank < keep) keys[rank] = sm.list[i];
        });
        if (tid == 0) p.counts[out] = min(n, keep);
    } else {
        uint64_t before = ~0ull;   // the key found last
        int found = 0;
        for (; found < keep; ++found) {
            uint64_t best = 0ull;
            for (uint32_t v = v0 + tid; v < v1; v += kNT) {
                float f[V];
                R::floats(x.load(v), f);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (f[i] > -INFINITY) {   // no NaN either
                        const uint64_t k = make_key(f[i], v * V + i);
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
    if (tid < lists) {
        sm.count[tid] = __ldcg(p.counts + list0 + tid);
        sm.mass[tid] = __ldcg(p.sums + list0 + tid);
    }
    __syncthreads();
    if (tid < p.n_beams) {
        Mass mass{-INFINITY, 0.0f};
        float top = -INFINITY;
        for (int l = tid * p.splits; l < (tid + 1) * p.splits; ++l) {
            mass = join(mass, Mass{sm.mass[l].x, sm.mass[l].y});
            if (sm.count[l] > 0) top = fmaxf(top, key_value(sm.cand[l * keep]));
        }
        const float cum = p.scores[seq * p.n_beams + tid];
        sm.top[tid] = top;
        sm.cum[tid] = cum;
        // log of the mass against the largest logit (its reference is no further than 16 below)
        const Wide l = wide_log(mass.sum), away = top == INFINITY ? Wide{0.0f, 0.0f} : two_sum(top, -mass.ref);
        sm.base[tid] = add(Wide{cum, 0.0f}, add(away, Wide{-l.hi, -l.lo}));
    }
    __syncthreads();
    if (tid == 0) {
        sm.floor = 0ull;
        sm.n_best = 0;
    }
    __syncthreads();
    // scores of all slices' elements.  The last of a full list has `keep` elements no worse than it: what
    // is worse than the best such is out
    const int n_cand = lists * keep;
    uint64_t floor = 0ull;
#pragma unroll 1
    for (int i = tid; i < n_cand; i += kNT) {
        const int list = i / keep, place = i - list * keep, beam = list / p.splits;
        uint64_t sc = 0ull;
        if (place < sm.count[list] && fabsf(sm.cum[beam]) <= kMaxF) {
            const float v = key_value(sm.cand[i]), top = sm.top[beam];
            // cum + (v - top) - log mass; what lies past f32 counts as its end (a mask's lowest value is
            // that, and goes on being told apart by the rest); nothing beside an infinite logit
            const auto end = [](Wide x) { return x.hi >= -kMaxF ? x : Wide{-kMaxF, 0.0f}; };
            const Wide d = v == top ? Wide{0.0f, 0.0f} : end(two_sum(v, -top));
            if (v == top || top < INFINITY) sc = ordered64(end(add(sm.base[beam], d)));
            if (place == keep - 1) floor = max(floor, sc);
        }
        sm.cand[i] = sc;   // its key is needed again by the few that stay: from global memory
    }
    if (floor) atomicMax(reinterpret_cast<unsigned long long*>(&sm.floor), (unsigned long long)floor);
    __syncthreads();
    floor = sm.floor;
    // what stays, in the lists' order
#pragma unroll 1
    for (int i0 = 0; i0 < n_cand; i0 += kNT) {
        const int i = i0 + tid;
        const uint64_t sc = i < n_cand ? sm.cand[i] : 0ull;
        const bool stays = sc != 0ull && sc >= floor;
        const unsigned who = __ballot_sync(kFull, stays);
        if (lane == 0) sm.warp_count[warp] = __popc(who);
        __syncthreads();
        int at = sm.n_best;
        for (int w = 0; w < warp; ++w) at += sm.warp_count[w];
        at += __popc(who & ((1u << lane) - 1u));
        if (stays) {
            sm.best[at] = sc;
            sm.best_at[at] = (uint16_t)i;
        }
        __syncthreads();
        if (tid == kNT - 1) sm.n_best = at + (stays ? 1 : 0);
        __syncthreads();
    }
    // by score, then the lower beam, then the key (a beam's score may be too large to tell its tokens apart)
    const int m = sm.n_best;
    float* os = p.out_scores + seq * keep;
    int32_t* op = p.parents + seq * keep;
    int32_t* ot = p.tokens + seq * keep;
    const uint64_t* all = p.keys + list0 * keep;
    const auto before = [&](int a, int b) {
        const int at_a = sm.best_at[a], at_b = sm.best_at[b];
        const int beam_a = at_a / keep / p.splits, beam_b = at_b / keep / p.splits;
        return beam_a != beam_b ? beam_a < beam_b : __ldcg(all + at_a) > __ldcg(all + at_b);
    };
    rank_all<true>(sm.best, m, before, [&](int i, int rank) {
        if (rank >= keep) return;
        const int at = sm.best_at[i];
        os[rank] = from_ordered((uint32_t)(sm.best[i] >> 32));
        op[rank] = (int32_t)(seq * p.n_beams + at / keep / p.splits);
        ot[rank] = (int32_t)key_index(__ldcg(all + at));
    });
    for (int k = m + tid; k < keep; k += kNT) {   // fewer continuations than asked for
        os[k] = -INFINITY;
        op[k] = -1;
        ot[k] = -1;
    }
}

// Slices of a row: 3 CTAs a SM at least, slices of at least 16 KB, lists within a request's limits.
constexpr int64_t kCtas = 152 * 3;
int64_t most_splits(int32_t n_beams, int64_t vocab, int32_t keep, int size) {
    const int64_t lists = std::min(kMaxLists / n_beams, kMaxCand / (n_beams * keep));
    return std::max<int64_t>(1, std::min(vocab * size / 16384, lists));
}
int splits_for(int64_t rows, int32_t n_beams, int64_t vocab, int32_t keep, int size) {
    return (int)std::min((kCtas + rows - 1) / std::max<int64_t>(1, rows), most_splits(n_beams, vocab, keep, size));
}
size_t round_up(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

// Tickets are zero between calls, so they have a place of their own whatever the sizes of the call.  Sized
// for either type (f32 rows have the most slices) and for fewer requests, of more slices each.
size_t beam_workspace_bytes(int32_t n_seq, int32_t n_beams, int64_t vocab, int32_t keep) {
    const int64_t rows = (int64_t)n_seq * n_beams;
    const int64_t lists = std::max(rows, std::min(rows + kCtas - 1, rows * most_splits(n_beams, vocab, keep, 4)));
    return kWsHeader + round_up(sizeof(uint32_t) * kBeamMaxSeq) + (size_t)lists * (sizeof(float2) + 8 * (size_t)keep + 4);
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
    p.per_split = (uint32_t)((vectors + p.splits - 1) / p.splits);
    p.scores = scores;
    p.out_scores = out_scores;
    p.parents = parents;
    p.tokens = tokens;
    char* ws = static_cast<char*>(workspace) + kWsHeader;
    p.tickets = reinterpret_cast<uint32_t*>(ws);
    ws += round_up(sizeof(uint32_t) * kBeamMaxSeq);
    p.sums = reinterpret_cast<float2*>(ws);
    p.keys = reinterpret_cast<uint64_t*>(p.sums + rows * p.splits);
    p.counts = reinterpret_cast<int32_t*>(p.keys + rows * p.splits * keep);
    const int64_t grid = rows * p.splits;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    return dt == KVQ_BF16 ? launch_chained(beam_select_kernel<__nv_bfloat16>, (unsigned)grid, kNT, 0, stream, p)
                          : launch_chained(beam_select_kernel<float>, (unsigned)grid, kNT, 0, stream, p);
}

}  // namespace kvq
