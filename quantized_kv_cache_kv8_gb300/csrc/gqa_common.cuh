// gqa_common.cuh -- what the grouped-query attention kernels share: the batch as the
// device sees it, the split of its work among the CTAs and the joining of cut tiles.
//
// Work.  For each sequence b and key-value head h there are n G query vectors, n the
// sequence's new tokens and G = n_heads / n_kv_heads (vector i G + g: token i, head
// h G + g).  They are cut into tiles of M; tile j needs
//   units(j) = max(1, ceil(limit(j) / N))
// steps of N rows, limit(j) the rows its last vector sees.  All steps of the batch,
// with OV more in front of each tile for its prologue, are numbered through, and CTA
// c of C takes the numbers [V c / C, V (c+1) / C): the same work for every CTA,
// whatever the lengths, and no length is read back by the host.  A tile that one CTA
// finishes is written at once; of a cut one, each CTA leaves its partial state
// in the workspace, and a second kernel joins the states, in the rows' order.  (Joined by
// the CTA that came last, 38 states of 16 x 256 took some 25 us.)
//
// The numbering needs sum_{i<j} units(i) in closed form.  Unmasked, units is the same
// for every tile.  Causal, with base = rows - n, for tiles with limit >= 1 but the last,
//   units(j) = floor((base + N + floor((M j + M - 1) / G)) / N) = floor((j + D) / R),
//   D = floor((G (base + N) + M - 1) / M),  R = G N / M
// (floors of quotients nest; M divides N): a sum of floors over consecutive integers.
#pragma once

#include "gqa.cuh"
#include "paged_common.cuh"
#include "tc_common.cuh"

namespace kvq {

struct GqaParams {
    int32_t n_seq, n_heads, n_kv, group, causal;
    const void* q;
    void* out;
    const uint8_t* k_codes;   // [n_pages][n_kv][page][D]
    const uint8_t* v_codes;
    const float2* scales;     // [n_pages][n_kv][page]
    const int64_t* cu_q;
    const int64_t* kv_lens;
    const int32_t* table;
    int32_t table_stride, shift, n_pages;
    int64_t max_tok;
    float sm_scale;
    int32_t* err;
    struct GqaCut* cuts;      // [CTAs]
    float2* ws_ml;            // [2 CTAs][M]
    float* ws_o;              // [2 CTAs][M * D], a kernel's own order
    float* ws_tot;            // tensor kernel: [CTAs][M * D], totals of long sums
    int64_t wait_limit, stall_polls;
};

struct GqaSeq {
    int32_t n, rows, base, tiles;
    int64_t q0, D, before, per_head;
    int64_t j0;
};
// The tile that a CTA begins and does not end: how many CTAs share it (0: there is none), where its outputs go.
struct alignas(16) GqaCut {
    int32_t count, h, vec0, vecs;
    int64_t q0;
};
// Part of a tile, as its CTA works on it (row counts fit 32 bits: a pool has fewer rows).
struct GqaSegment {
    int32_t b, h;
    int32_t vec0;           // vector 0 of the tile, within (sequence, kv head)
    int32_t vecs;           // vectors of the tile
    int32_t base, rows;     // token i sees base + 1 + i rows (causal) or all of them
    int32_t limit;          // rows the tile's last vector sees
    int32_t u0, u1;
    int32_t last;           // the CTA's last
    int32_t first, count;   // of a cut tile: the first CTA that holds steps of it, and how many do
    int32_t slot;           // where this CTA leaves its state of it; -1: the tile is whole
    int64_t q0;             // the sequence's first token
};

// A CTA's walk over its segments, by one warp (the others read the segment from shared memory: the
// walk would cost every thread 40 registers, and each line of its code may have to be fetched).
// What only batches with several tiles a head need stands in functions of its own.
// LEAST: numbers a CTA takes at least, so that few long tiles are not cut into more states than
// their joining is worth.
template <int M, int N, int OV, int LEAST>
struct GqaWalk {
    static_assert(N % M == 0, "closed form");
    int64_t v_end, per;          // the CTA's last number + 1; numbers a CTA
    int32_t extra, ctas, c;      // CTAs with one number more; CTAs that hold any; this one
    int32_t b, h, j;             // sequence, kv head, tile
    int64_t seq_v;               // the sequence's first number
    GqaSeq s;
    int64_t u0;

    __device__ __forceinline__ static GqaSeq shape(const GqaParams& p, int b) {
        GqaSeq s{0, 0, 0, 0, 0, 0, 0, 0, 0};
        if (b >= p.n_seq) return s;
        const int64_t a = p.cu_q[b], e = p.cu_q[b + 1];
        int64_t kv = p.kv_lens[b];
        // a table row, and the pool, hold so many rows; row indices stay within int32
        const int64_t cap = min((int64_t)min(p.table_stride, p.n_pages) << p.shift, (int64_t)0x7fffffff - 1024);
        if (a < 0 || e < a || e > p.max_tok || kv < 0 || kv > cap) set_err(p.err, KVQ_ERR_ARG);
        if (a < 0 || e <= a || e > p.max_tok) return s;
        kv = min(max(kv, (int64_t)0), cap);
        s.q0 = a;
        s.n = (int32_t)(e - a);
        s.rows = (int32_t)kv;
        s.base = (int32_t)(kv - s.n);
        s.tiles = (int32_t)(((int64_t)s.n * p.group + M - 1) / M);
        // the last tile's last vector is the last token's, which sees every row
        const int64_t last = OV + max(1, (s.rows + N - 1) / N);
        s.per_head = s.tiles == 1 ? last : many(p, s) + last;
        return s;
    }
    // Numbers of a head before its last tile; fills in the closed form.
    __device__ __noinline__ static int64_t many(const GqaParams& p, GqaSeq& s) {
        if (p.causal) {
            const int64_t G = p.group, base = s.base;
            s.j0 = base >= 0 ? 0 : (-base * G) / M;   // first tile with limit >= 1
            const int64_t C = G * (base + N) + M - 1;
            s.D = C >= 0 ? C / M : -((-C + M - 1) / M);
            s.before = floor_sum(p, s.j0 + s.D);
        }
        return prefix_many(p, s, s.tiles - 1);
    }
    __device__ __noinline__ static int64_t floor_sum(const GqaParams& p, int64_t n) {   // sum_{k<n} floor(k / R)
        const int64_t R = (int64_t)p.group * (N / M), q = quot(n, R), r = n - q * R;
        return R * (q * (q - 1) / 2) + q * r;
    }
    // Numbers of a head before tile j (j < tiles).
    __device__ __noinline__ static int64_t prefix_many(const GqaParams& p, const GqaSeq& s, int64_t j) {
        if (!p.causal) return j * (OV + max(1, (s.rows + N - 1) / N));
        const int64_t v = OV * j + min(j, s.j0);
        return j <= s.j0 ? v : v + floor_sum(p, j + s.D) - s.before;
    }
    __device__ __forceinline__ static int64_t prefix(const GqaParams& p, const GqaSeq& s, int64_t j) {
        return j == 0 ? 0 : prefix_many(p, s, j);
    }
    // Rows that the last vector of tile j sees.
    __device__ __forceinline__ static int32_t limit(const GqaParams& p, const GqaSeq& s, int32_t j) {
        if (!p.causal || j == s.tiles - 1) return s.rows;
        return max(0, s.base + 1 + (int32_t)((uint32_t)(M * j + M - 1) / (uint32_t)p.group));
    }
    __device__ __forceinline__ int64_t start_of(int64_t k) const { return k * per + min(k, (int64_t)extra); }
    // CTA of number v
    __device__ __forceinline__ int32_t cta_of(int64_t v) const {
        const int64_t big = (int64_t)extra * (per + 1);
        return (int32_t)(v < big ? quot(v, per + 1) : extra + quot(v - big, per));
    }
    // The numbers dealt out, this CTA's share; false when it has none.
    __device__ __forceinline__ bool deal(int64_t sum, int32_t k, int32_t n_cta) {
        c = k;
        ctas = (int32_t)min((int64_t)n_cta, (sum + LEAST - 1) / LEAST);
        if (c >= ctas) return false;
        per = quot(sum, ctas);
        extra = (int32_t)(sum - per * ctas);
        v_end = start_of(c + 1);
        return true;
    }
    // The place of number v in sequence b (its shape in s, first number in seq_v), by whole warps: 32 tiles are
    // tried at a time.
    __device__ __forceinline__ void place(const GqaParams& p, int64_t v) {
        int64_t x = v - seq_v;
        h = x < s.per_head ? 0 : (int32_t)quot(x, s.per_head);
        x -= h * s.per_head;
        int32_t lo = 0, hi = s.tiles;
        while (hi - lo > 1) {
            const int32_t step = (hi - lo + 31) / 32;
            const int64_t mid = lo + (int64_t)step * (1 + (int32_t)(threadIdx.x & 31));
            const bool before = mid < hi && prefix_many(p, s, mid) <= x;
            lo += step * __popc(__ballot_sync(kFull, before));
            hi = (int32_t)min((int64_t)hi, (int64_t)lo + step);
        }
        j = lo;
        u0 = max((int64_t)0, x - prefix(p, s, lo) - OV);
    }
    // By one warp, for batches of up to kFew sequences.  False when CTA k has nothing to do.
    static constexpr int kFew = 256;
    __device__ __forceinline__ bool start_few(const GqaParams& p, int32_t k, int32_t n_cta) {
        const int lane = threadIdx.x & 31;
        GqaSeq y = shape(p, lane);
        int64_t mine = y.per_head * p.n_kv;
#pragma unroll 1
        for (int i = lane + 32; i < p.n_seq; i += 32) mine += shape(p, i).per_head * p.n_kv;
        int64_t sum = mine;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        if (!deal(sum, k, n_cta)) return false;
        const int64_t v0 = start_of(c);
        int64_t first = 0;
#pragma unroll 1
        for (int k0 = 0;; k0 += 32) {
            if (k0 > 0) y = shape(p, k0 + lane);
            const int64_t n = y.per_head * p.n_kv;
            int64_t incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t t = __shfl_up_sync(kFull, incl, o);
                if (lane >= o) incl += t;
            }
            const unsigned who = __ballot_sync(kFull, v0 >= first + incl - n && v0 < first + incl);
            if (who) {
                const int l = __ffs(who) - 1;
                b = k0 + l;
                seq_v = __shfl_sync(kFull, first + incl - n, l);
                s.n = __shfl_sync(kFull, y.n, l);
                s.rows = __shfl_sync(kFull, y.rows, l);
                s.base = __shfl_sync(kFull, y.base, l);
                s.tiles = __shfl_sync(kFull, y.tiles, l);
                s.q0 = __shfl_sync(kFull, y.q0, l);
                s.D = __shfl_sync(kFull, y.D, l);
                s.before = __shfl_sync(kFull, y.before, l);
                s.per_head = __shfl_sync(kFull, y.per_head, l);
                s.j0 = __shfl_sync(kFull, y.j0, l);
                break;
            }
            first += __shfl_sync(kFull, incl, 31);
        }
        place(p, v0);
        return true;
    }
    // By all NT threads of the CTA, any number of sequences; part: 2 NT / 32 int64s, found: 2.
    template <int NT>
    __device__ __noinline__ bool start_many(const GqaParams& p, int32_t k, int32_t n_cta, int64_t* part, int64_t* found) {
        const int tid = threadIdx.x;
        int64_t all = 0, incl, sum;
        for (int i = tid; i < p.n_seq; i += NT) all += shape(p, i).per_head * p.n_kv;
        block_scan<NT>(all, part, &sum);
        if (!deal(sum, k, n_cta)) return false;   // every thread alike
        const int64_t v0 = start_of(c);
        int64_t first = 0;
        for (int k0 = 0; k0 < p.n_seq; k0 += NT) {
            const int64_t n = shape(p, k0 + tid).per_head * p.n_kv;
            incl = block_scan<NT>(n, part, &sum);
            if (v0 >= first + incl - n && v0 < first + incl) {
                found[0] = k0 + tid;
                found[1] = first + incl - n;
            }
            first += sum;
            if (v0 < first) break;
        }
        __syncthreads();
        b = (int32_t)found[0];
        seq_v = found[1];
        s = shape(p, b);
        place(p, v0);
        return true;
    }
    // The current segment; false past the CTA's last.
    __device__ __forceinline__ bool get(const GqaParams& p, GqaSegment& g) const {
        const int64_t tile_v = seq_v + h * s.per_head + prefix(p, s, j);
        const int32_t lim = limit(p, s, j), n = max(1, (lim + N - 1) / N);
        const int64_t end = v_end - tile_v - OV;
        const int32_t u1 = (int32_t)min((int64_t)n, end);
        if (u1 <= u0) return false;
        g.b = b;
        g.h = h;
        g.limit = lim;
        g.u0 = (int32_t)u0;
        g.u1 = u1;
        g.last = end <= n;
        g.q0 = s.q0;
        g.vec0 = M * j;
        g.vecs = (int32_t)min((int64_t)M, (int64_t)s.n * p.group - (int64_t)M * j);
        g.base = s.base;
        g.rows = s.rows;
        g.slot = -1;
        if (u0 > 0 || u1 < n) {
            // a CTA begins at most one tile that it does not end, and ends one that it did not begin
            g.first = u0 == 0 ? c : cta_of(tile_v + OV);
            g.count = (u1 == n ? c : cta_of(tile_v + OV + n - 1)) - g.first + 1;
            g.slot = slot(c, g.first);
        }
        return true;
    }
    // On to the next tile, by a whole warp (sequences without new tokens are passed 32 at a time).
    // False past the CTA's last.
    __device__ __forceinline__ bool next(const GqaParams& p) {
        u0 = 0;
        if (++j < s.tiles) return true;
        j = 0;
        if (++h < p.n_kv) return true;
        h = 0;
        seq_v += s.per_head * p.n_kv;
        if (seq_v >= v_end) return false;
        for (++b; b < p.n_seq; b += 32) {
            const int k = b + (int)(threadIdx.x & 31);
            bool some = false;
            if (k < p.n_seq) {
                const int64_t a = p.cu_q[k], e = p.cu_q[k + 1];
                some = a >= 0 && e > a && e <= p.max_tok;
            }
            const unsigned hit = __ballot_sync(kFull, some);
            if (hit == 0u) continue;
            b += __ffs(hit) - 1;
            s = shape(p, b);
            return true;
        }
        return false;
    }
    // Where a CTA leaves its state of a tile: its own begun and not ended, or the end of another's.
    __device__ static int32_t slot(int32_t k, int32_t first) { return k == first ? 2 * k + 1 : 2 * k; }
};

// Rows that vector v (within its sequence and kv head) sees.
__device__ __forceinline__ int32_t gqa_limit(const GqaParams& p, const GqaSegment& g, int32_t v) {
    return p.causal ? max(0, g.base + 1 + (int32_t)((uint32_t)v / (uint32_t)p.group)) : g.rows;
}
// Element offset of vector v in q and out.
template <int D>
__device__ __forceinline__ int64_t gqa_vector(const GqaParams& p, const GqaSegment& g, int32_t v) {
    const int32_t tok = (int32_t)((uint32_t)v / (uint32_t)p.group);
    return ((g.q0 + tok) * p.n_heads + g.h * p.group + (v - tok * p.group)) * (int64_t)D;
}
// Page that holds row t of sequence b; a table
// entry outside the pool sets the error word and reads page 0 instead.
__device__ __forceinline__ int32_t gqa_page(const GqaParams& p, int32_t b, int32_t t) {
    int32_t id = p.table[(int64_t)b * p.table_stride + (t >> p.shift)];
    if (id < 0 || id >= p.n_pages) {
        set_err(p.err, KVQ_ERR_ARG);
        id = 0;
    }
    return id;
}

// A key's scale as its scores take it: NaN for an infinite one (0 times it is NaN), whose row a negative
// product would hide.
__device__ __forceinline__ float key_scale(float s) { return __fmaf_rn(s, 0.0f, s); }

// What the scores of a vector held as 2^-e of itself are multiplied by: binades.  NaN for a vector with an infinity,
// whose scores of -inf would hide rows.
__device__ __forceinline__ float query_scale(float sm_scale, int e, float amax) {
    return sm_scale * tc::kLog2e * __uint_as_float((uint32_t)(127 + e) << 23) * __fmaf_rn(amax, 0.0f, 1.0f);
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }

// The tensor-core kernel (gqa_tc.cu): f32 queries up to 128 dims.
size_t gqa_tc_state_bytes(int32_t head_dim);
bool gqa_tc_supported(int32_t head_dim, kvq_dtype dt);
cudaError_t launch_gqa_tc(const GqaParams& p, int32_t head_dim, kvq_dtype dt, void* state, cudaStream_t stream);

constexpr int kGqaMaxCtas = 760;
constexpr size_t kGqaCutBytes = kGqaMaxCtas * sizeof(GqaCut);

}  // namespace kvq
