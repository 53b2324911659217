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
    int64_t q0, n, base, rows, tiles, j0, D, before, per_head;
};
// The tile that a CTA begins and does not end: how many CTAs share it (0: there is none), where its outputs go.
struct GqaCut {
    int32_t count, h, vec0, vecs;
    int64_t q0;
    int64_t pad;
};
// Part of a tile, as its CTA works on it (row counts fit 32 bits: a pool has fewer rows).
struct GqaSegment {
    int32_t b, h;
    int32_t vec0;           // vector 0 of the tile, within (sequence, kv head)
    int32_t vecs;           // vectors of the tile
    int32_t base, rows;     // token i sees base + 1 + i rows (causal) or all of them
    int32_t limit;          // rows the tile's last vector sees
    int32_t u0, u1, units;
    int32_t first, count;   // of a cut tile: the first CTA that holds steps of it, and how many do
    int32_t slot;           // where this CTA leaves its state of it; -1: the tile is whole
    int64_t q0;             // the sequence's first token
};

template <int M, int N, int OV>
struct GqaWalk {
    static_assert(N % M == 0, "closed form");
    template <int NT>
    static constexpr int kScratch = NT / 32 + 2 + sizeof(GqaSeq) / 8;
    int64_t v_end, total, ctas, c;
    int32_t b;
    int64_t x;        // h * tiles + j of the current tile
    int64_t seq_v;
    GqaSeq s;
    int64_t u0;

    __device__ __noinline__ static GqaSeq shape(const GqaParams& p, int b) {
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
        s.n = e - a;
        s.rows = kv;
        s.base = kv - s.n;
        s.tiles = (s.n * p.group + M - 1) / M;
        if (p.causal) {
            const int64_t G = p.group;
            s.j0 = s.base >= 0 ? 0 : (-s.base * G) / M;   // first tile with limit >= 1
            const int64_t C = G * (s.base + N) + M - 1;
            s.D = C >= 0 ? C / M : -((-C + M - 1) / M);
            s.before = floor_sum(p, s.j0 + s.D);
        }
        s.per_head = prefix(p, s, s.tiles - 1) + OV + units(p, s, s.tiles - 1);
        return s;
    }
    // rows that the last vector of tile j sees
    __device__ static int64_t limit(const GqaParams& p, const GqaSeq& s, int64_t j) {
        if (!p.causal) return s.rows;
        return max((int64_t)0, s.base + 1 + min(s.n - 1, quot(M * j + M - 1, p.group)));
    }
    __device__ static int64_t units(const GqaParams& p, const GqaSeq& s, int64_t j) {
        return max((int64_t)1, (limit(p, s, j) + N - 1) / N);
    }
    __device__ __noinline__ static int64_t floor_sum(const GqaParams& p, int64_t n) {   // sum_{k<n} floor(k / R)
        const int64_t R = (int64_t)p.group * (N / M), q = quot(n, R), r = n - q * R;
        return R * (q * (q - 1) / 2) + q * r;
    }
    // numbers of a head before tile j (j < tiles)
    __device__ static int64_t prefix(const GqaParams& p, const GqaSeq& s, int64_t j) {
        if (!p.causal) return j * (OV + max((int64_t)1, (s.rows + N - 1) / N));
        const int64_t v = OV * j + min(j, s.j0);
        return j <= s.j0 ? v : v + floor_sum(p, j + s.D) - s.before;
    }
    __device__ __forceinline__ int64_t start_of(int64_t k) const { return quot(total * k, ctas); }
    // CTA of number v
    __device__ __forceinline__ int64_t cta_of(int64_t v) const {
        int64_t k = quot(v * ctas, total);
        while (start_of(k + 1) <= v) ++k;
        while (start_of(k) > v) --k;
        return k;
    }

    // By all NT threads; part: kScratch<NT> int64s.  False when CTA k has nothing to do.
    template <int NT>
    __device__ __forceinline__ bool start(const GqaParams& p, int64_t k, int64_t n_cta, int64_t* part) {
        const int tid = threadIdx.x;
        c = k;
        total = 0;
        GqaSeq y;
        int64_t n = 0, incl = 0, sum = 0, v0 = 0, first = 0;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
            for (int k0 = 0; k0 < p.n_seq; k0 += NT) {
                if (pass == 0 || p.n_seq > NT) {   // a batch of at most NT sequences is read once
                    y = shape(p, k0 + tid);
                    n = y.per_head * p.n_kv;
                    incl = block_scan<NT>(n, part, &sum);
                }
                if (pass == 0) {
                    total += sum;
                    continue;
                }
                if (v0 >= first + incl - n && v0 < first + incl) {
                    GqaSeq* own = reinterpret_cast<GqaSeq*>(part + NT / 32 + 2);
                    *own = y;
                    part[NT / 32] = k0 + tid;
                    part[NT / 32 + 1] = first + incl - n;
                }
                first += sum;
                if (v0 < first) break;
            }
            if (pass == 0) {
                ctas = min(n_cta, total);
                if (c >= ctas) return false;   // every thread alike
                v0 = start_of(c);
                v_end = start_of(c + 1);
            }
        }
        __syncthreads();
        b = (int32_t)part[NT / 32];
        seq_v = part[NT / 32 + 1];
        s = *reinterpret_cast<const GqaSeq*>(part + NT / 32 + 2);
        const int64_t h = quot(v0 - seq_v, s.per_head), v = v0 - seq_v - h * s.per_head;
        int64_t lo = 0, hi = s.tiles;
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) / 2;
            if (prefix(p, s, mid) <= v) lo = mid;
            else hi = mid;
        }
        x = h * s.tiles + lo;
        u0 = max((int64_t)0, v - prefix(p, s, lo) - OV);
        return true;
    }
    // The current segment; false past the CTA's last.
    __device__ __noinline__ bool get(const GqaParams& p, GqaSegment& g) const {
        if (b >= p.n_seq) return false;
        const int64_t h = quot(x, s.tiles), j = x - h * s.tiles;
        const int64_t tile_v = seq_v + h * s.per_head + prefix(p, s, j), lim = limit(p, s, j);
        const int64_t n = max((int64_t)1, (lim + N - 1) / N), u1 = min(n, v_end - tile_v - OV);
        if (u1 <= u0) return false;
        g.b = b;
        g.h = (int32_t)h;
        g.limit = (int32_t)lim;
        g.units = (int32_t)n;
        g.u0 = (int32_t)u0;
        g.u1 = (int32_t)u1;
        g.q0 = s.q0;
        g.vec0 = (int32_t)(M * j);
        g.vecs = (int32_t)min((int64_t)M, s.n * p.group - M * j);
        g.base = (int32_t)s.base;
        g.rows = (int32_t)s.rows;
        g.slot = -1;
        if (u0 > 0 || u1 < n) {
            // a CTA begins at most one tile that it does not end, and ends one that it did not begin
            g.first = (int32_t)(u0 == 0 ? c : cta_of(tile_v + OV));
            g.count = (int32_t)cta_of(tile_v + OV + n - 1) - g.first + 1;
            g.slot = slot((int32_t)c, g.first);
        }
        return true;
    }
    // On to the next tile, by whole warps (sequences without new tokens are passed 32 at a time).
    __device__ __noinline__ void next(const GqaParams& p) {
        u0 = 0;
        if (++x < s.tiles * p.n_kv) return;
        seq_v += s.per_head * p.n_kv;
        x = 0;
        ++b;
        if (seq_v >= v_end) b = p.n_seq;   // the rest is for the CTAs after this one
        for (; b < p.n_seq; b += 32) {
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
            return;
        }
    }
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

// The tensor-core kernel (gqa_tc.cu): f32 queries up to 128 dims.
size_t gqa_tc_state_bytes(int32_t head_dim);
bool gqa_tc_supported(int32_t head_dim, kvq_dtype dt);
cudaError_t launch_gqa_tc(const GqaParams& p, int32_t head_dim, kvq_dtype dt, void* state, cudaStream_t stream);

constexpr int kGqaMaxCtas = 760;
constexpr size_t kGqaCutBytes = kGqaMaxCtas * sizeof(GqaCut);

}  // namespace kvq
