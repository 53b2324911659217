// paged_common.cuh -- what the paged attention kernels share: the batch as the
// device sees it, the split of its work among the CTAs, the partial states and
// the lookup of a row's place in the pool.
//
// Work.  Sequence b has n = cu_q[b+1] - cu_q[b] new tokens and kv_lens[b] rows
// in its pages, the new ones included; token i sees the rows [0, base + i + 1),
// base = kv_lens[b] - n.  Its n * H query vectors (token-major, as they lie in
// memory) are cut into tiles of M; tile j needs
//   units(j) = max(1, ceil(limit(j) / N)),  limit(j) = base + 1 + token of its last vector
// steps of N rows (N a multiple of M).  All steps of the batch, with kOverhead
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
//            = floor((j + D) / (k H)),  D = floor((H (base + N) + M - 1) / M), k = N / M
// (floors of quotients nest), a sum of floors over consecutive integers.
#pragma once

#include "attn_common.cuh"

namespace kvq {

struct PagedParams {
    int32_t n_seq, n_heads;
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
    SignWords signs;
    float kn[2];
    float lv[16];
};

// Quotient of non-negative integers: a 64-bit division takes some hundred
// instructions, and nearly every one of these fits 32 bits.
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
    if (((uint64_t)a | (uint64_t)b) >> 32) return a / b;
    return (int64_t)((uint32_t)a / (uint32_t)b);
}

struct SeqShape {
    int64_t q0, n_new, base, tiles, j0, D;
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
    static constexpr int64_t kRatio = N / M;
    static constexpr int kLogM = M == 32 ? 5 : 7, kLogN = N == 32 ? 5 : 7;
    static_assert((1 << kLogM) == M && (1 << kLogN) == N, "tile sizes");

    __device__ static SeqShape shape(const PagedParams& p, int b) {
        SeqShape s{0, 0, 0, 0, 0, 0};
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
        return s;
    }
    __device__ static int64_t units(const SeqShape& s, int64_t H, int64_t j) {
        const int64_t tok = min(s.n_new - 1, quot(M * j + M - 1, H));
        return max((int64_t)1, (s.base + tok + N) >> kLogN);
    }
    __device__ static int64_t floor_sum(int64_t n, int64_t d) {   // sum_{k<n} floor(k / d)
        const int64_t q = quot(n, d), r = n - q * d;
        return d * (q * (q - 1) / 2) + q * r;
    }
    // numbers before tile j (j < tiles)
    __device__ static int64_t prefix(const SeqShape& s, int64_t H, int64_t j) {
        const int64_t v = OV * j + min(j, s.j0), d = kRatio * H;
        return j <= s.j0 ? v : v + floor_sum(j + s.D, d) - floor_sum(s.j0 + s.D, d);
    }
    __device__ static int64_t total(const SeqShape& s, int64_t H) {
        if (s.tiles == 0) return 0;
        return prefix(s, H, s.tiles - 1) + OV + units(s, H, s.tiles - 1);
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
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        const int64_t x = part[w];
        before += w < warp ? x : 0;
        all += x;
    }
    *sum = all;
    return v + before;
}

// A CTA's walk over its segments.  start() is called by all NT threads of the
// CTA; the rest by any thread on its own (every thread holds the same walk).
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
        const int64_t H = p.n_heads;
        // batches of at most NT sequences: one thread each, read once
        SeqShape x = S::shape(p, tid);
        int64_t n = S::total(x, H), mine = n, sum;
        for (int k = tid + NT; k < p.n_seq; k += NT) mine += S::total(S::shape(p, k), H);
        int64_t incl = block_scan<NT>(mine, part, &sum);
        total = sum;
        ctas = min(n_cta, total);
        if (c >= ctas) return false;   // every thread alike
        const int64_t v0 = start_of(c);
        v_end = start_of(c + 1);
        int64_t base = 0;
        for (int k0 = 0; k0 < p.n_seq; k0 += NT) {
            if (p.n_seq > NT) {
                x = S::shape(p, k0 + tid);
                n = S::total(x, H);
                incl = base + block_scan<NT>(n, part, &sum);
            }
            if (v0 >= incl - n && v0 < incl) {
                part[NT / 32] = k0 + tid;
                part[NT / 32 + 1] = incl - n;
            }
            base += sum;
            if (v0 < base) break;
        }
        __syncthreads();
        b = (int32_t)part[NT / 32];
        seq_v = part[NT / 32 + 1];
        s = S::shape(p, b);
        int64_t lo = 0, hi = s.tiles;
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) / 2;
            if (S::prefix(s, H, mid) <= v0 - seq_v) lo = mid;
            else hi = mid;
        }
        j = lo;
        u0 = max((int64_t)0, v0 - seq_v - S::prefix(s, H, j) - (int64_t)overhead());
        return true;
    }
    __device__ static constexpr int overhead() { return S::kOverhead; }

    // The current segment; false past the CTA's last.
    __device__ __forceinline__ bool get(const PagedParams& p, Segment& g) const {
        if (b >= p.n_seq) return false;
        const int64_t H = p.n_heads;
        g.b = b;
        g.tile_v = seq_v + S::prefix(s, H, j);
        g.units = S::units(s, H, j);
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
    __device__ __forceinline__ void next(const PagedParams& p) {
        u0 = 0;
        if (++j < s.tiles) return;
        seq_v += S::total(s, p.n_heads);
        j = 0;
        do {
            s = S::shape(p, ++b);
        } while (b < p.n_seq && s.tiles == 0);
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
__device__ __forceinline__ int64_t row_limit(const Segment& g, int r, int n_heads) {
    return max((int64_t)0, g.base + 1 + quot(g.tok0 + r, n_heads));
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

// The exact (fp32) kernel and the tensor-core kernel: query vectors a tile,
// rows a step, prologue allowance in steps; CTAs, and pairs of CTAs, that walk.
using PagedSimt = SchedOf<32, 32, 4>;
using PagedTensor = SchedOf<128, 128, 2>;
constexpr int kPagedCtas = 152, kPagedPairs = 76;

cudaError_t launch_paged_tensor(kvq_format fmt, const PagedParams& p, cudaStream_t stream);

}  // namespace kvq
