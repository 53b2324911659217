// paged_common.cuh -- what the paged attention kernels share: the batch as the
// device sees it, the split of its work among the CTAs, the partial states and
// the lookup of a row's place in the pool.
//
// Work.  Sequence b has n = cu_q[b+1] - cu_q[b] new tokens and kv_lens[b] rows
// in its pages, the new ones included; token i sees the rows [0, base + i + 1),
// base = kv_lens[b] - n.  Its n * H query vectors (token-major, as they lie in
// memory) are cut into tiles of M; tile j needs
//   units(j) = max(1, ceil(limit(j) / N)),  limit(j) = base + 1 + token of its last vector
// steps of N rows (N = M).  All steps of the batch, with kOverhead
// more in front of each tile for its prologue, are numbered through, and CTA c
// of C takes the numbers [V c / C, V (c+1) / C): every CTA gets the same work
// whatever the lengths, a long sequence is spread over many CTAs, and nothing
// is read back by the host.  A tile that one CTA finishes is written at once;
// a cut tile leaves partial states (at most two per CTA: the end of a tile
// begun before it, the beginning of one it does not end), which the merge
// kernel joins.
//
// The numbering needs sum_{i<j} units(i) in closed form.  Where limit >= 1 and j
// is not the last tile,
//   units(j) = floor((base + N + floor((M j + M - 1) / H)) / N)
//            = floor((H (base + N) + M j + M - 1) / (N H))
//            = floor((j + D) / H),  D = floor((H (base + N) + M - 1) / M), as M = N
// (floors of quotients nest), a sum of floors over consecutive integers.
#pragma once

#include "paged.cuh"

namespace kvq {

struct PagedParams {
    int32_t n_seq, n_heads;
    uint64_t h_inv;            // floor((2^64 - 1) / n_heads)
    const void* q;             // [tokens][n_heads][576]
    void* out;                 // [tokens][n_heads][512], the query's type
    const uint8_t* codes;
    const float* scales;
    const int64_t* cu_q;
    const int64_t* kv_lens;
    const int32_t* table;
    int32_t table_stride, shift, n_pages, n_blocks;
    int64_t max_tok;           // query tokens the caller passed
    float sm_scale;
    int32_t* err;
    uint32_t* exact_count;
    int64_t wait_limit, stall_polls;
    float* ws_o;               // [2 * CTAs][M][512]
    float* ws_ml;              // [2 * CTAs][M][2]
    int64_t* ws_desc;          // [CTAs][4]: parts, first query vector, vectors
    float2* ws_l;              // tensor kernel: [CTAs][256 threads], totals of long sums
    float* ws_c;               // exact kernel: [CTAs][M][512], what the totals rounded away
    SignWords signs;
    float kn[2];
    float lv[16];
};

// Quotients of non-negative integers.  By the head count: a multiplication with
// h_inv = floor((2^64 - 1) / n_heads), at most 1 short, then a correction (inlined
// 64-bit divisions made the walk 80 KB of code, fetched anew by every launch).  By
// anything else, out of line.
__device__ __forceinline__ int64_t over_heads(const PagedParams& p, int64_t n) {
    int64_t q = (int64_t)__umul64hi((uint64_t)n, p.h_inv);
    if (n - q * p.n_heads >= p.n_heads) ++q;
    return q;
}
static __device__ __noinline__ int64_t quot(int64_t a, int64_t b) {
    if (((uint64_t)a | (uint64_t)b) >> 32) return a / b;
    return (int64_t)((uint32_t)a / (uint32_t)b);
}

struct SeqShape {
    int64_t q0, n_new, base, tiles, j0, D;
    int64_t before;    // sum_{k < j0 + D} floor(k / H)
};
struct Segment {
    int32_t b;
    int64_t row0;      // first query vector of the tile, in the whole batch
    int32_t rows;      // query vectors of the tile
    int64_t tok0;      // token (within the sequence) of vector 0, times H plus head: M j
    int64_t base, n_new;
    int64_t u0, u1, units;
    int64_t tile_v;    // the tile's first number
};

template <int M, int N, int OV>
struct PagedSched {
    static constexpr int kM = M, kN = N;
    static_assert(M == N, "the closed form below is for steps of as many rows as a tile has vectors");
    static constexpr int kLogM = M == 32 ? 5 : 7, kLogN = N == 32 ? 5 : 7;
    static_assert((1 << kLogM) == M && (1 << kLogN) == N, "tile sizes");

    // does sequence b have new tokens (and valid offsets)?
    __device__ static bool some(const PagedParams& p, int b) {
        if (b >= p.n_seq) return false;
        const int64_t a = p.cu_q[b], e = p.cu_q[b + 1];
        return a >= 0 && e > a && e <= p.max_tok;
    }
    __device__ static SeqShape shape(const PagedParams& p, int b) {
        SeqShape s{0, 0, 0, 0, 0, 0, 0};
        if (b >= p.n_seq) return s;
        const int64_t a = p.cu_q[b], e = p.cu_q[b + 1];
        int64_t kv = p.kv_lens[b];
        // a table row, and the pool, hold so many rows; row indices stay within int32
        const int64_t cap = min((int64_t)min(p.table_stride, p.n_pages) << p.shift, (int64_t)0x7fffffff - 1024);
        if (a < 0 || e < a || e > p.max_tok || kv < 0 || kv > cap) set_err(p.err, KVQ_ERR_ARG);
        if (a < 0 || e <= a || e > p.max_tok) return s;
        kv = min(max(kv, (int64_t)0), cap);
        const int64_t H = p.n_heads;
        s.q0 = a;
        s.n_new = e - a;
        s.base = kv - s.n_new;
        s.tiles = (s.n_new * H + M - 1) >> kLogM;
        s.j0 = s.base >= 0 ? 0 : (-s.base * H) >> kLogM;   // first tile with limit >= 1
        const int64_t C = H * (s.base + N) + M - 1;
        s.D = C >> kLogM;   // floor, also below zero
        s.before = floor_sum(p, s.j0 + s.D);
        return s;
    }
    __device__ static int64_t units(const PagedParams& p, const SeqShape& s, int64_t j) {
        const int64_t tok = min(s.n_new - 1, over_heads(p, M * j + M - 1));
        return max((int64_t)1, (s.base + tok + N) >> kLogN);
    }
    __device__ static int64_t floor_sum(const PagedParams& p, int64_t n) {   // sum_{k<n} floor(k / H)
        const int64_t H = p.n_heads, q = over_heads(p, n), r = n - q * H;
        return H * (q * (q - 1) / 2) + q * r;
    }
    // numbers before tile j (j < tiles)
    __device__ static int64_t prefix(const PagedParams& p, const SeqShape& s, int64_t j) {
        const int64_t v = OV * j + min(j, s.j0);
        return j <= s.j0 ? v : v + floor_sum(p, j + s.D) - s.before;
    }
    __device__ static int64_t total(const PagedParams& p, const SeqShape& s) {
        if (s.tiles == 0) return 0;
        return prefix(p, s, s.tiles - 1) + OV + units(p, s, s.tiles - 1);
    }
};

// Sum of v over the CTA's NT threads and this thread's inclusive prefix.
template <int NT>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* part, int64_t* sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += t;
    }
    __syncthreads();
    if (lane == 31) part[warp] = v;
    __syncthreads();
    int64_t w = lane < NT / 32 ? part[lane] : 0;   // every warp scans the warps' sums
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(kFull, w, o);
        if (lane >= o) w += t;
    }
    *sum = __shfl_sync(kFull, w, NT / 32 - 1);
    const int64_t before = __shfl_sync(kFull, w, max(warp - 1, 0));
    return warp > 0 ? v + before : v;
}

// Scratch of start() in int64s: the warps' sums, the found sequence.
template <int NT>
constexpr int kWalkScratch = NT / 32 + 9;

// A CTA's walk over its segments.  start() is called by all NT threads of the
// CTA, next() by whole warps; the rest by any thread on its own (every thread holds
// the same walk).
template <class S>
struct PagedWalk {
    int64_t v_end, total, ctas;   // the CTA's last number + 1; numbers in all; CTAs that hold any
    int32_t b;
    int64_t j, seq_v;             // tile within the sequence; the sequence's first number
    SeqShape s;
    int64_t u0;

    __device__ __forceinline__ int64_t start_of(int64_t c) const { return quot(total * c, ctas); }

    // False when this CTA has nothing to do.
    template <int NT>
    __device__ __forceinline__ bool start(const PagedParams& p, int64_t c, int64_t n_cta, int64_t* part) {
        const int tid = threadIdx.x;
        SeqShape x;
        int64_t n = 0, incl = 0, sum = 0, v0 = 0, base = 0;
        total = 0;
        // pass 0 adds up the numbers, pass 1 finds this CTA's first; a batch of at
        // most NT sequences, a thread each, is read once
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
            for (int k0 = 0; k0 < p.n_seq; k0 += NT) {
                if (pass == 0 || p.n_seq > NT) {
                    x = S::shape(p, k0 + tid);
                    n = S::total(p, x);
                    incl = block_scan<NT>(n, part, &sum);
                }
                if (pass == 0) {
                    total += sum;
                    continue;
                }
                if (v0 >= base + incl - n && v0 < base + incl) {
                    int64_t* own = part + NT / 32;
                    own[0] = k0 + tid;
                    own[1] = base + incl - n;
                    own[2] = x.q0;
                    own[3] = x.n_new;
                    own[4] = x.base;
                    own[5] = x.tiles;
                    own[6] = x.j0;
                    own[7] = x.D;
                    own[8] = x.before;
                }
                base += sum;
                if (v0 < base) break;
            }
            if (pass == 0) {
                ctas = min(n_cta, total);
                if (c >= ctas) return false;   // every thread alike
                v0 = start_of(c);
                v_end = start_of(c + 1);
            }
        }
        __syncthreads();
        const int64_t* own = part + NT / 32;
        b = (int32_t)own[0];
        seq_v = own[1];
        s = SeqShape{own[2], own[3], own[4], own[5], own[6], own[7], own[8]};
        int64_t lo = 0, hi = s.tiles;
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) / 2;
            if (S::prefix(p, s, mid) <= v0 - seq_v) lo = mid;
            else hi = mid;
        }
        j = lo;
        u0 = max((int64_t)0, v0 - seq_v - S::prefix(p, s, j) - (int64_t)overhead());
        return true;
    }
    __device__ static constexpr int overhead() { return S::kOverhead; }

    // The current segment; false past the CTA's last.
    __device__ __forceinline__ bool get(const PagedParams& p, Segment& g) const {
        if (b >= p.n_seq) return false;
        const int64_t H = p.n_heads;
        g.b = b;
        g.tile_v = seq_v + S::prefix(p, s, j);
        g.units = S::units(p, s, j);
        g.u0 = u0;
        g.u1 = min(g.units, v_end - g.tile_v - overhead());
        if (g.u1 <= g.u0) return false;
        g.row0 = s.q0 * H + S::kM * j;
        g.rows = (int32_t)min((int64_t)S::kM, s.n_new * H - S::kM * j);
        g.tok0 = S::kM * j;
        g.base = s.base;
        g.n_new = s.n_new;
        return true;
    }
    // On to the next, by a whole warp: past sequences without new tokens (a padded
    // batch has long runs of them) 32 at a time.
    __device__ __forceinline__ void next(const PagedParams& p) {
        u0 = 0;
        if (++j < s.tiles) return;
        seq_v += S::total(p, s);
        j = 0;
        ++b;
        if (seq_v >= v_end) b = p.n_seq;   // the rest is for the walkers after this one
        for (; b < p.n_seq; b += 32) {
            const unsigned hit = __ballot_sync(kFull, S::some(p, b + (int)(threadIdx.x & 31)));
            if (hit == 0u) continue;
            b += __ffs(hit) - 1;
            s = S::shape(p, b);
            return;
        }
    }
    // CTA of number v
    __device__ __forceinline__ int64_t cta_of(int64_t v) const {
        int64_t c = quot(v * ctas, total);
        while (start_of(c + 1) <= v) ++c;
        while (start_of(c) > v) --c;
        return c;
    }
    // Where a segment that does not span its tile leaves its state (-1: it
    // spans it): slot 2 c for the end of a tile begun earlier, 2 c + 1 for the
    // beginning of one that goes on; parts = CTAs that share the tile then.
    __device__ __forceinline__ int64_t slot(const Segment& g, int64_t c, int64_t* parts) const {
        *parts = 0;
        if (g.u0 == 0 && g.u1 == g.units) return -1;
        if (g.u0 > 0) return 2 * c;
        *parts = cta_of(g.tile_v + overhead() + g.units - 1) - c + 1;
        return 2 * c + 1;
    }
};

template <int M, int N, int OV>
struct SchedOf : PagedSched<M, N, OV> {
    static constexpr int kOverhead = OV;
};

// Rows query vector r of a segment sees (r counts within the tile).
__device__ __forceinline__ int64_t row_limit(const PagedParams& p, const Segment& g, int r) {
    return max((int64_t)0, g.base + 1 + over_heads(p, g.tok0 + r));
}

// Pool row of row t of sequence b; a table entry outside the pool sets the
// error word and reads page 0 instead.
__device__ __forceinline__ int32_t paged_row(const PagedParams& p, int32_t b, int64_t t) {
    int32_t id = p.table[(int64_t)b * p.table_stride + (t >> p.shift)];
    if (id < 0 || id >= p.n_pages) {
        set_err(p.err, KVQ_ERR_ARG);
        id = 0;
    }
    return (id << p.shift) + (int32_t)(t & ((1ll << p.shift) - 1));
}

// A row's scales as the kernels use them.  One that is no finite number makes the
// row's score NaN, and counts through it alone, where the mask can drop it: as a
// weight's factor it would be 0 x NaN for the tokens that do not see the row.
__device__ __forceinline__ float2 row_scales(float latent, float rope) {
    const bool ok = fmaxf(fabsf(latent), fabsf(rope)) <= 3.402823466e38f && latent == latent && rope == rope;
    return ok ? make_float2(latent, rope) : make_float2(0.0f, __uint_as_float(0x7fffffffu));
}

// The exact (fp32) kernel and the tensor-core kernel: query vectors a tile,
// rows a step, prologue allowance in steps (the exact kernel: 16 sequences of 60 to
// 1000 rows x 32 heads 44 us with 4, 46 with 2, 59 with 8; the tensor kernel: first
// chunk of 777 in 4 bits 320 us with 4, 362 with 2, 341 with 6, mixed 24 sequences
// 206, 218, 211); CTAs, and pairs of CTAs, that walk.
using PagedSimt = SchedOf<32, 32, 4>;
using PagedTensor = SchedOf<128, 128, 4>;
constexpr int kPagedCtas = 152, kPagedPairs = 76;

cudaError_t launch_paged_tensor(kvq_format fmt, const PagedParams& p, cudaStream_t stream);

}  // namespace kvq
