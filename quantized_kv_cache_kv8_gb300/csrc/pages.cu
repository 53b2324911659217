// pages.cu -- block tables and slot maps of a paged row pool, built on the GPU
// from the lengths of a batch's requests.
//
// A pool of n_pages pages of P = 2^shift rows; sequence s holds
// ceil(len_s / P) pages, listed in row s of the block table.  With n_s new rows:
//   old_s = ceil(len_s / P), tot_s = ceil((len_s + n_s) / P), need_s = tot_s - old_s
//   off_s = sum_{r < s} need_r, cu_s = sum_{r < s} n_r
//   page j < need_s of sequence s  <-  free[n_free - 1 - (off_s + j)]
//   slot of new row i of s         =   page(len_s + i) * P + (len_s + i) mod P
// and the trim back to k_s rows puts page c (ceil(k_s / P) <= c < ceil(len_s / P))
// at free[n_free + total - 1 - rank], rank its place in (sequence, page) order:
// the inverse of the reservation, so a step that is taken back leaves the free
// list as it was.
//
// What bounds it: a decode step moves a few KB, so the call is one launch and
// one chain of dependent reads (lengths, the scan, the table entry or the free
// list, the slot).  Every CTA therefore scans all the lengths itself, up to 1024 at
// a time, instead of waiting for another launch's prefix sums; it then writes its
// share of the rows (a binary search over the scanned offsets in shared
// memory) and of the new table entries.  The counters that are both read and
// written (n_free, and the lengths where the caller updates them in place) are
// written by the CTA that arrives last, after every read.  A trim writes the pages
// above the stack's top first: where one of them is no page, that CTA, which has heard
// of it with the arrivals, leaves the top and the lengths as they were.
// Measured, a reservation and its trim in a replayed graph: 64 sequences of one new
// row 5.7 us, 1024 sequences of up to 63 12.1 us.
#include "paged.cuh"

#include <algorithm>

namespace kvq {
namespace {

constexpr int kSmall = 256, kLarge = 1024;   // threads of a CTA = sequences scanned at once
constexpr int64_t kMaxLen = 1ll << 40;
constexpr uint32_t kBadTicket = 1u << 16;    // arrivals below it, CTAs with a broken entry above

struct PagesParams {
    int32_t n_seq, shift, table_stride, n_pages;
    const int64_t* lens;
    const int64_t* arg;      // reserve: new rows; trim: rows to keep
    int32_t* table;
    int32_t* free_pages;
    int32_t* n_free;
    int64_t* lens_out;
    int64_t* cu_new;
    int64_t* slots;
    int64_t* positions;
    int64_t max_new;
    int32_t* err;
    uint32_t* ticket;
};

__device__ __forceinline__ int64_t pages_of(int64_t rows, int shift) {
    return (rows + ((1ll << shift) - 1)) >> shift;
}

// Inclusive scan of two values over the CTA (kNT threads); totals in tot[2].
template <int kNT>
__device__ __forceinline__ void block_scan2(int64_t& a, int64_t& b, int64_t (*part)[2], int64_t* tot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t ta = __shfl_up_sync(kFull, a, o), tb = __shfl_up_sync(kFull, b, o);
        if (lane >= o) {
            a += ta;
            b += tb;
        }
    }
    __syncthreads();   // part and tot may still be read by the previous scan's users
    if (lane == 31) {
        part[warp][0] = a;
        part[warp][1] = b;
    }
    __syncthreads();
    if (warp == 0) {
        int64_t pa = lane < kNT / 32 ? part[lane][0] : 0, pb = lane < kNT / 32 ? part[lane][1] : 0;
#pragma unroll
        for (int o = 1; o < kNT / 32; o <<= 1) {
            const int64_t ta = __shfl_up_sync(kFull, pa, o), tb = __shfl_up_sync(kFull, pb, o);
            if (lane >= o) {
                pa += ta;
                pb += tb;
            }
        }
        if (lane < kNT / 32) {
            part[lane][0] = pa;
            part[lane][1] = pb;
        }
        if (lane == kNT / 32 - 1) {
            tot[0] = pa;
            tot[1] = pb;
        }
    }
    __syncthreads();
    if (warp > 0) {
        a += part[warp - 1][0];
        b += part[warp - 1][1];
    }
}

struct SeqNeed {
    int64_t len, rows;    // cached rows; rows added (reserve) or kept (trim)
    int32_t p0, p1;       // the pages [p0, p1) taken or given back
    bool bad;
};

template <bool TRIM>
__device__ __forceinline__ SeqNeed seq_need(const PagesParams& p, int s) {
    SeqNeed r{0, 0, 0, 0, false};
    if (s >= p.n_seq) return r;
    const int64_t len = p.lens[s], arg = p.arg[s];
    if (len < 0 || len > kMaxLen || (!TRIM && (arg < 0 || arg > kMaxLen))) {
        r.bad = true;
        return r;
    }
    const int64_t keep = (arg < 0 || arg > len) ? len : arg;
    const int64_t lo = pages_of(TRIM ? keep : len, p.shift), hi = pages_of(TRIM ? len : len + arg, p.shift);
    if (hi > p.table_stride) {
        r.bad = true;
        return r;
    }
    r.len = len;
    r.rows = TRIM ? keep : arg;
    r.p0 = (int32_t)lo;
    r.p1 = (int32_t)hi;
    return r;
}

// Largest i in [0, n) with off[i] <= x (off ascending, off[0] = 0 <= x).
__device__ __forceinline__ int find_last(const int32_t* off, int n, int32_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <bool TRIM, int kNT>
__global__ void __launch_bounds__(kNT) pages_kernel(PagesParams p) {
    __shared__ int64_t part[kNT / 32][2], tot[2];
    __shared__ int64_t s_len[kNT];
    __shared__ int32_t s_row[kNT], s_page[kNT], s_p0[kNT];   // s_row, s_page: exclusive prefixes within the chunk
    __shared__ int s_last, s_bad;
    launch_dependents();
    grid_dependency_wait();
    const int tid = threadIdx.x;
    const int64_t G = gridDim.x, c = blockIdx.x;
    const int n_chunks = (p.n_seq + kNT - 1) / kNT;
    const int32_t n_free = *p.n_free;

    // totals and checks over the whole batch, by every CTA alike
    int64_t rows = 0, pages = 0;
    bool bad = false;
    SeqNeed one{};
    for (int k = 0; k < n_chunks; ++k) {
        one = seq_need<TRIM>(p, k * kNT + tid);
        rows += TRIM ? 0 : one.rows;
        pages += one.p1 - one.p0;
        bad |= one.bad;
    }
    bad = __syncthreads_or(bad);
    int64_t row_incl = rows, page_incl = pages;
    block_scan2<kNT>(row_incl, page_incl, part, tot);
    const int64_t row_total = tot[0], page_total = tot[1];
    int status = KVQ_OK;
    if (bad || n_free < 0 || n_free > p.n_pages || row_total > p.max_new) status = KVQ_ERR_ARG;
    else if (TRIM ? page_total > p.n_pages - n_free : page_total > n_free) status = TRIM ? KVQ_ERR_ARG : KVQ_ERR_WORKSPACE;

    if (status != KVQ_OK) {
        // all or nothing: no page moves, every slot is refused
        if (c == 0 && tid == 0 && p.err) atomicCAS(p.err, 0, status);
        if (!TRIM) {
            for (int64_t i = c * kNT + tid; i < p.max_new; i += G * kNT) {
                p.slots[i] = -1;
                if (p.positions) p.positions[i] = 0;
            }
            for (int64_t s = c * kNT + tid; s <= p.n_seq; s += G * kNT) p.cu_new[s] = 0;
            for (int64_t s = c * kNT + tid; s < p.n_seq; s += G * kNT) p.lens_out[s] = p.lens[s];
        }
        return;
    }

    if (!TRIM && c == 0 && tid == 0) p.cu_new[0] = 0;
    // this CTA's rows, a contiguous share of the slot map
    const int64_t per = (p.max_new + G - 1) / G;
    const int64_t r0 = min(c * per, p.max_new), r1 = min(r0 + per, p.max_new);
    const int64_t mask = (1ll << p.shift) - 1;
    const int64_t top = (int64_t)n_free - 1;
    bool bad_page = false;
    int64_t row_base = 0, page_base = 0;
    for (int k = 0; k < n_chunks; ++k) {
        const int s = k * kNT + tid;
        int64_t ri = row_incl, pi = page_incl;   // the totals' scan is the only chunk's
        if (n_chunks > 1) {
            one = seq_need<TRIM>(p, s);
            ri = TRIM ? 0 : one.rows;
            pi = one.p1 - one.p0;
            block_scan2<kNT>(ri, pi, part, tot);
        }
        const int64_t chunk_rows = tot[0], chunk_pages = tot[1];
        s_len[tid] = one.len;
        s_row[tid] = (int32_t)(ri - (TRIM ? 0 : one.rows));
        s_page[tid] = (int32_t)(pi - (one.p1 - one.p0));
        s_p0[tid] = one.p0;
        __syncthreads();
        const int live = min(kNT, p.n_seq - k * kNT);
        if (!TRIM) {
            if (c == 0) {
                if (s < p.n_seq) p.cu_new[s + 1] = row_base + ri;
            }
            const int64_t a = max(r0, row_base), b = min(r1, row_base + chunk_rows);
            for (int64_t i = a + tid; i < b; i += kNT) {
                const int32_t x = (int32_t)(i - row_base);
                const int q = find_last(s_row, live, x);
                const int64_t pos = s_len[q] + (x - s_row[q]);
                const int64_t pg = pos >> p.shift;
                const int32_t id = pg < s_p0[q] ? p.table[(int64_t)(k * kNT + q) * p.table_stride + pg]
                                                : p.free_pages[top - (page_base + s_page[q] + (pg - s_p0[q]))];
                const bool ok = id >= 0 && id < p.n_pages;
                bad_page |= !ok;
                p.slots[i] = ok ? ((int64_t)id << p.shift) + (pos & mask) : -1;
                if (p.positions) p.positions[i] = pos;
            }
        }
        for (int64_t e = c * kNT + tid; e < chunk_pages; e += G * kNT) {
            const int q = find_last(s_page, live, (int32_t)e);
            const int64_t rank = page_base + e;
            int32_t* entry = p.table + (int64_t)(k * kNT + q) * p.table_stride + s_p0[q] + (e - s_page[q]);
            if (TRIM) {
                const int32_t id = *entry;
                bad_page |= id < 0 || id >= p.n_pages;
                p.free_pages[top + page_total - rank] = id;
            } else {
                *entry = p.free_pages[top - rank];
            }
        }
        row_base += chunk_rows;
        page_base += chunk_pages;
        __syncthreads();
    }
    if (!TRIM)
        for (int64_t i = max(r0, row_total) + tid; i < r1; i += kNT) {   // rows past the batch: no slot
            p.slots[i] = -1;
            if (p.positions) p.positions[i] = 0;
        }
    if (bad_page && p.err) atomicCAS(p.err, 0, (int32_t)KVQ_ERR_ARG);

    // the last CTA to get here updates what the others have read
    bad_page = __syncthreads_or(bad_page);
    if (G > 1) {
        if (tid == 0) {
            __threadfence();
            const uint32_t before = atomicAdd(p.ticket, bad_page ? kBadTicket + 1u : 1u);
            s_last = (before & (kBadTicket - 1u)) == (uint32_t)(G - 1);
            s_bad = bad_page || before >= kBadTicket;
            __threadfence();
        }
        __syncthreads();
        if (!s_last) return;
        bad_page = s_bad;
        if (tid == 0) *p.ticket = 0u;
    }
    if (TRIM && bad_page) return;
    for (int s = tid; s < p.n_seq; s += kNT) {
        const SeqNeed r = n_chunks > 1 ? seq_need<TRIM>(p, s) : one;
        p.lens_out[s] = TRIM ? r.rows : r.len + r.rows;
    }
    if (tid == 0) *p.n_free = n_free + (int32_t)(TRIM ? page_total : -page_total);
}

PagesParams base_params(int32_t n_seq, int32_t page_rows, const int64_t* lens, const int64_t* arg, int32_t* table,
                        int32_t table_stride, int32_t* free_pages, int32_t* n_free, int32_t n_pages, void* workspace) {
    PagesParams p{};
    p.n_seq = n_seq;
    while ((1 << p.shift) < page_rows) ++p.shift;
    p.table_stride = table_stride;
    p.n_pages = n_pages;
    p.lens = lens;
    p.arg = arg;
    p.table = table;
    p.free_pages = free_pages;
    p.n_free = n_free;
    p.err = static_cast<int32_t*>(workspace);
    p.ticket = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + 4);
    return p;
}

}  // namespace

cudaError_t launch_pages_reserve(int32_t n_seq, int32_t page_rows, const int64_t* lens, const int64_t* new_lens,
                                 int32_t* table, int32_t table_stride, int32_t* free_pages, int32_t* n_free,
                                 int32_t n_pages, int64_t* lens_out, int64_t* cu_new, int64_t* slots,
                                 int64_t* positions, int64_t max_new, void* workspace, cudaStream_t stream) {
    PagesParams p = base_params(n_seq, page_rows, lens, new_lens, table, table_stride, free_pages, n_free, n_pages,
                                workspace);
    p.lens_out = lens_out;
    p.cu_new = cu_new;
    p.slots = slots;
    p.positions = positions;
    p.max_new = max_new;
    // about two rows a thread: one CTA (no ticket) for a decode step's rows
    if (n_seq <= kSmall && max_new <= 2 * kSmall) {
        return launch_chained(pages_kernel<false, kSmall>, 1, kSmall, 0, stream, p);
    } else {
        const int64_t grid = std::min<int64_t>(152, std::max<int64_t>(1, (max_new + 2 * kLarge - 1) / (2 * kLarge)));
        return launch_chained(pages_kernel<false, kLarge>, (unsigned)grid, kLarge, 0, stream, p);
    }
}

cudaError_t launch_pages_trim(int32_t n_seq, int32_t page_rows, int64_t* lens, const int64_t* keep, int32_t* table,
                              int32_t table_stride, int32_t* free_pages, int32_t* n_free, int32_t n_pages,
                              void* workspace, cudaStream_t stream) {
    PagesParams p =
        base_params(n_seq, page_rows, lens, keep, table, table_stride, free_pages, n_free, n_pages, workspace);
    p.lens_out = lens;
    if (n_seq <= kSmall) return launch_chained(pages_kernel<true, kSmall>, 1, kSmall, 0, stream, p);
    return launch_chained(pages_kernel<true, kLarge>, (unsigned)std::min(8, (n_seq + kLarge - 1) / kLarge), kLarge, 0, stream,
                          p);
}

}  // namespace kvq
