// fork.cu -- block tables that follow the parents chosen by a beam search: sequences
// share their parents' full pages, and pages that nobody holds any more return to the
// stack of free pages.
//
// Sequence i continues the rows of sequence f = parents[i] (-1: it ends).  Of f's
// ceil(len / P) pages the full ones are listed by every child.  The page in progress
// (len mod P rows of it) stays with f's first child; every other child gets a free page
// and an entry (from, to) in the list of copies, which pages_copy carries out on the
// pools of all layers.  So rows are only ever appended to pages that one sequence holds.
// Which pages are let go needs no counts beside the tables: a page is free when each of
// the sequences that held it has no child.
//
//   1  marks[page] = kept for the pages of sequences with children; the other sequences s
//      raise it to n - s at least: where no child holds the page, its lowest holder owns it
//   2  the new table rows, from the old ones, and the owned pages go into the workspace
//   3  the rows go into the table, the owned pages onto the stack in (sequence, page) order;
//      marks are cleared, lengths and the free count written
//
// What bounds it: the latency of these dependent passes; the tables of a batch are a few
// hundred KB.  One cluster of 8 CTAs does it in one launch, with a cluster barrier
// between passes; its 256 warps take pieces of 128 pages of a sequence in turn.  512 sequences of 53
// pages on average take 17.5 us, 64 of 36 10.9 (with each piece's sequence found by bisection 20.1 and
// 11.4; by a CTA that takes one sequence after another 79 for the 512).
#include "gqa.cuh"

#include <algorithm>
#include <cooperative_groups.h>

namespace kvq {
namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8, kNT = 1024, kWarps = kNT / 32;
constexpr int kMaxSeq = 4096;
constexpr int kPiece = 128, kPer = kPiece / 32;   // pages of a piece, of a lane
constexpr int32_t kKept = 0x7fffffff;
constexpr int64_t kMaxLen = 1ll << 40;

struct ForkParams {
    int32_t n_seq, shift, stride, n_pages;
    const int32_t* parents;
    int64_t* lens;
    int32_t* table;
    int32_t* free_pages;
    int32_t* n_free;
    int32_t* copies;
    int32_t* err;
    int32_t* marks;     // [n_pages], zero between calls
    int32_t* rows;      // [n_seq][stride], the new table
    int32_t* gone;      // [n_seq][stride], owned pages, from the start of each piece
    int32_t* counts;    // [pieces], how many
    int32_t* places;    // [pieces], how many before them
};

struct ForkShared {
    int32_t first[kMaxSeq];       // a sequence's first child, n_seq without one
    int32_t pages[kMaxSeq];       // pages of it
    int32_t piece0[kMaxSeq + 1];  // pieces of the sequences before it
    int32_t rank[kMaxSeq];        // of sequence i: copies before it, or -1
    int32_t parent[kMaxSeq];
    int2 gone[kNT];               // of the first kNT pieces: owned pages, of the pieces before
    uint16_t of[kNT];             // and their sequences
    int64_t part[kWarps];
    int bad;
    int32_t flag;                 // this CTA met a page outside the pool
};

__device__ __forceinline__ void set_copy(const ForkParams& p, int i, int32_t from, int32_t to) {
    p.copies[2 * i] = from;   // aligned to its elements only
    p.copies[2 * i + 1] = to;
}

// Exclusive scan over the CTA of one value a thread; the total in *sum.
__device__ __forceinline__ int64_t scan(int64_t v, int64_t* part, int64_t* sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += t;
    }
    __syncthreads();
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    int64_t w = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(kFull, w, o);
        if (lane >= o) w += t;
    }
    *sum = __shfl_sync(kFull, w, 31);
    const int64_t before = __shfl_sync(kFull, w, max(warp - 1, 0));
    return incl - v + (warp > 0 ? before : 0);
}

__device__ __forceinline__ int find_last(const int32_t* off, int n, int32_t x) {   // largest i < n with off[i] <= x
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// A warp's piece: pages [w0, w0 + kPiece) of sequence s; lane l holds w0 + l, w0 + l + 32, ...
struct Piece {
    int s, w0, pages;
    __device__ __forceinline__ Piece(const ForkShared& sm, int n, int32_t k)
        : s(k < kNT ? sm.of[k] : find_last(sm.piece0, n, k)), w0((k - sm.piece0[s]) * kPiece), pages(sm.pages[s]) {}
    __device__ __forceinline__ void load(const int32_t* table, int32_t stride, int lane, int32_t (&id)[kPer]) const {
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int w = w0 + 32 * u + lane;
            id[u] = w < pages ? __ldcg(table + (int64_t)s * stride + w) : -1;
        }
    }
};

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kNT, 1) pages_fork_kernel(ForkParams p) {
    extern __shared__ __align__(16) unsigned char raw[];
    ForkShared& sm = *reinterpret_cast<ForkShared*>(raw);
    cg::cluster_group cluster = cg::this_cluster();
    launch_dependents();
    grid_dependency_wait();
    const int tid = threadIdx.x, lane = tid & 31, n = p.n_seq;
    const int cta = (int)cluster.block_rank(), gw = (tid >> 5) * kCluster + cta;   // warp of the cluster
    const int32_t P = 1 << p.shift;
    const int32_t n_free = __ldcg(p.n_free);
    // the batch, by every CTA alike
    if (tid == 0) {
        sm.bad = n_free < 0 || n_free > p.n_pages;
        sm.flag = 0;
    }
    for (int i = tid; i < n; i += kNT) sm.first[i] = n;
    __syncthreads();
    int32_t parent[kMaxSeq / kNT];
    bool whole[kMaxSeq / kNT];
    int64_t len[kMaxSeq / kNT];   // of the parents: the new lengths
#pragma unroll
    for (int k = 0; k < kMaxSeq / kNT; ++k) {
        const int i = k * kNT + tid;
        parent[k] = -1;
        if (i < n) {
            const int32_t f = __ldcg(p.parents + i);
            const int64_t len = __ldcg(p.lens + i), pages = (len + P - 1) >> p.shift;
            if (f < -1 || f >= n || len < 0 || len > kMaxLen || pages > p.stride) {
                sm.bad = 1;
            } else {
                parent[k] = f;
                sm.pages[i] = (int32_t)pages;
                if (f >= 0) atomicMin(&sm.first[f], i);
            }
            sm.parent[i] = parent[k];
            sm.rank[i] = (len & (P - 1)) != 0;   // until the ranks are known: a page in progress
        }
    }
    __syncthreads();
    const bool bad = sm.bad != 0;
#pragma unroll
    for (int k = 0; k < kMaxSeq / kNT; ++k) {
        whole[k] = parent[k] < 0 || sm.rank[parent[k]] == 0;
        len[k] = cta == 0 && parent[k] >= 0 ? __ldcg(p.lens + parent[k]) : 0;
    }
    __syncthreads();
    int32_t pieces = 0, copies = 0;
    if (!bad) {
#pragma unroll
        for (int k = 0; k < kMaxSeq / kNT; ++k) {
            if (k * kNT >= n) break;
            const int i = k * kNT + tid;
            const int32_t f = parent[k];
            const bool copy = !whole[k] && sm.first[f] != i;
            int64_t sum;
            const int64_t at =
                scan(((int64_t)(i < n ? (sm.pages[i] + kPiece - 1) / kPiece : 0) << 32) + copy, sm.part, &sum);
            if (i < n) {
                const int32_t k0 = pieces + (int32_t)(at >> 32), k1 = min(k0 + (sm.pages[i] + kPiece - 1) / kPiece, kNT);
                sm.piece0[i] = k0;
                for (int32_t j = k0; j < k1; ++j) sm.of[j] = (uint16_t)i;
                sm.rank[i] = copy ? copies + (int32_t)(uint32_t)at : -1;
            }
            pieces += (int32_t)(sum >> 32);
            copies += (int32_t)(uint32_t)sum;
        }
        if (tid == 0) sm.piece0[n] = pieces;
    }
    __syncthreads();
    const int32_t status = bad ? KVQ_ERR_ARG : copies > n_free ? KVQ_ERR_WORKSPACE : KVQ_OK;
    const int stride_w = kCluster * kWarps;
    if (status == KVQ_OK) {
        bool wrong = false;
        for (int32_t k = gw; k < pieces; k += stride_w) {
            const Piece q(sm, n, k);
            int32_t id[kPer];
            q.load(p.table, p.stride, lane, id);
            const bool kept = sm.first[q.s] < n;
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                if (q.w0 + 32 * u + lane >= q.pages) continue;
                if (id[u] < 0 || id[u] >= p.n_pages) wrong = true;
                else if (kept) p.marks[id[u]] = kKept;
                else atomicMax(p.marks + id[u], n - q.s);   // below kKept, whichever comes first
            }
        }
        // the pages that copies take
        for (int32_t i = cta * kNT + tid; i < copies; i += kCluster * kNT) {
            const int32_t id = __ldcg(p.free_pages + n_free - 1 - i);
            if (id < 0 || id >= p.n_pages) wrong = true;
        }
        if (wrong) sm.flag = 1;
    }
    cluster.sync();
    bool broken = status != KVQ_OK;
    for (int r = 0; r < kCluster; ++r) broken |= *cluster.map_shared_rank(&sm.flag, r) != 0;
    if (!broken) {
        for (int32_t k = gw; k < pieces; k += stride_w) {
            const Piece q(sm, n, k);
            int32_t owned = 0;
            if (sm.first[q.s] >= n) {
                int32_t id[kPer], mark[kPer];
                q.load(p.table, p.stride, lane, id);
#pragma unroll
                for (int u = 0; u < kPer; ++u) mark[u] = id[u] >= 0 ? __ldcg(p.marks + id[u]) : 0;
#pragma unroll
                for (int u = 0; u < kPer; ++u) {
                    const bool own = id[u] >= 0 && mark[u] == n - q.s;
                    const unsigned who = __ballot_sync(kFull, own);
                    if (own) p.gone[(int64_t)q.s * p.stride + q.w0 + owned + __popc(who & ((1u << lane) - 1u))] = id[u];
                    owned += __popc(who);
                }
            }
            if (lane == 0) p.counts[k] = owned;
        }
        // new rows, a piece of the parent's a warp at a time
        for (int i = gw; i < n; i += stride_w) {
            const int32_t f = sm.parent[i];
            if (f < 0) continue;
            const int32_t pages = sm.pages[f], rank = sm.rank[i];
            const int32_t to = rank >= 0 ? __ldcg(p.free_pages + n_free - 1 - rank) : 0;
            const int32_t* src = p.table + (int64_t)f * p.stride;
            int32_t* dst = p.rows + (int64_t)i * p.stride;
#pragma unroll 4
            for (int32_t w = lane; w < pages; w += 32) {
                int32_t id = __ldcg(src + w);
                if (rank >= 0 && w == pages - 1) {
                    set_copy(p, i, id, to);
                    id = to;
                }
                dst[w] = id;
            }
        }
    }
    cluster.sync();
    // every CTA adds up what the pieces let go
    const bool few = pieces <= kNT;
    int64_t total = 0;
    if (!broken) {
        if (few) {
            const int32_t c = tid < pieces ? __ldcg(p.counts + tid) : 0;
            const int64_t at = scan(c, sm.part, &total);
            sm.gone[tid] = make_int2(c, (int32_t)at);
            __syncthreads();
        } else {
            int64_t freed = 0;
            for (int32_t k0 = 0; k0 < pieces; k0 += kNT) freed += k0 + tid < pieces ? __ldcg(p.counts + k0 + tid) : 0;
            scan(freed, sm.part, &total);
        }
    }
    const int64_t top = (int64_t)n_free - copies + total;
    broken |= top > p.n_pages;   // a page listed twice by a sequence
    if (broken) {
        if (status == KVQ_OK)   // marks of the pages that are some
            for (int32_t k = gw; k < pieces; k += stride_w) {
                const Piece q(sm, n, k);
                int32_t id[kPer];
                q.load(p.table, p.stride, lane, id);
#pragma unroll
                for (int u = 0; u < kPer; ++u)
                    if (id[u] >= 0 && id[u] < p.n_pages) p.marks[id[u]] = 0;
            }
        if (cta == 0 && tid == 0 && p.err) atomicCAS(p.err, 0, status != KVQ_OK ? status : (int32_t)KVQ_ERR_ARG);
        for (int i = cta * kNT + tid; i < n; i += kCluster * kNT)
            set_copy(p, i, -1, -1);
        return;
    }
    // owned pages onto the stack, a piece a warp, from the place its counts before it give
    if (!few) {
        int64_t base = 0;
        for (int32_t k0 = 0; k0 < pieces; k0 += kNT) {
            const int32_t k = k0 + tid;
            int64_t sum;
            const int64_t at = base + scan(k < pieces ? __ldcg(p.counts + k) : 0, sm.part, &sum);
            base += sum;
            if (k < pieces && k % kCluster == cta) p.places[k] = (int32_t)at;   // this CTA's warps'
        }
        __syncthreads();
    }
    for (int32_t k = gw; k < pieces; k += stride_w) {
        const int2 c = few ? sm.gone[k] : make_int2(__ldcg(p.counts + k), __ldcg(p.places + k));
        if (c.x == 0) continue;
        const Piece q(sm, n, k);
        const int32_t* src = p.gone + (int64_t)q.s * p.stride + q.w0;
        const int64_t last = top - 1 - c.y;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int j = 32 * u + lane;
            if (j < c.x) {
                const int32_t id = __ldcg(src + j);
                p.marks[id] = 0;
                p.free_pages[last - j] = id;
            }
        }
    }
    if (cta == 0 && tid == 0) *p.n_free = (int32_t)top;
    if (cta == 0) {   // the other CTAs are past their reads
#pragma unroll
        for (int k = 0; k < kMaxSeq / kNT; ++k) {
            const int i = k * kNT + tid;
            if (i < n) p.lens[i] = len[k];
        }
    }
    for (int i = gw; i < n; i += stride_w) {
        const int32_t f = sm.parent[i];
        if (lane == 0 && sm.rank[i] < 0) set_copy(p, i, -1, -1);
        if (f < 0) continue;
        const int32_t pages = sm.pages[f];
        const int32_t* src = p.rows + (int64_t)i * p.stride;
        int32_t* dst = p.table + (int64_t)i * p.stride;
#pragma unroll 4
        for (int32_t w = lane; w < pages; w += 32) {
            const int32_t id = __ldcg(src + w);
            dst[w] = id;
            p.marks[id] = 0;   // every page that was kept is some child's
        }
    }
}

constexpr int kCopyNT = 256, kCopyPer = 4, kMaxPools = 128;

struct CopyParams {
    const int32_t* copies;
    int32_t n_pages, n_pools;
    int32_t* err;
    kvq_pool pool[kMaxPools];
    uint32_t unit0[kMaxPools + 1];   // units of a page in the pools before it
};

// Unit: the type that pages are moved in.  A page's units in all pools are numbered through; a
// CTA moves 1024 of them, so small arrays (scales) share one.  What bounds it: memory; 8 layers'
// pages of 16 rows, 2 heads of 256, for 270 of 512 children: 14 us, 5.1 TB/s (as much with the
// copies picked out first and taken in turn by 608 CTAs).
template <typename Unit>
__global__ void __launch_bounds__(kCopyNT) pages_copy_kernel(const __grid_constant__ CopyParams p) {
    launch_dependents();
    grid_dependency_wait();
    const int i = blockIdx.x;
    const int32_t from = __ldcg(p.copies + 2 * i), to = __ldcg(p.copies + 2 * i + 1);
    if (from < 0 || to < 0) return;
    if (from >= p.n_pages || to >= p.n_pages) {
        if (threadIdx.x == 0 && p.err) atomicCAS(p.err, 0, (int32_t)KVQ_ERR_ARG);
        return;
    }
    const uint32_t units = p.unit0[p.n_pools];
    for (uint64_t y = blockIdx.y; y * (kCopyNT * kCopyPer) < units; y += gridDim.y) {
        Unit v[kCopyPer];
        Unit* dst[kCopyPer];
#pragma unroll
        for (int u = 0; u < kCopyPer; ++u) {
            const uint64_t x = y * (kCopyNT * kCopyPer) + u * kCopyNT + threadIdx.x;
            dst[u] = nullptr;
            if (x < units) {
                int lo = 0, hi = p.n_pools;
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (p.unit0[mid] <= x) lo = mid;
                    else hi = mid;
                }
                char* base = static_cast<char*>(p.pool[lo].data);
                const int64_t at = (int64_t)(x - p.unit0[lo]) * sizeof(Unit), bytes = p.pool[lo].page_bytes;
                v[u] = *reinterpret_cast<const Unit*>(base + from * bytes + at);
                dst[u] = reinterpret_cast<Unit*>(base + to * bytes + at);
            }
        }
#pragma unroll
        for (int u = 0; u < kCopyPer; ++u)
            if (dst[u]) *dst[u] = v[u];
    }
}

template <typename Unit>
cudaError_t launch_copy(CopyParams& p, int32_t n, cudaStream_t stream) {
    uint64_t units = 0;
    for (int32_t k = 0; k < p.n_pools; ++k) {
        p.unit0[k] = (uint32_t)units;
        units += p.pool[k].page_bytes / sizeof(Unit);
        if (units > 0x7fffffff) return cudaErrorInvalidConfiguration;
    }
    p.unit0[p.n_pools] = (uint32_t)units;
    if (units == 0) return cudaSuccess;
    const unsigned y = (unsigned)std::min<uint64_t>((units + kCopyNT * kCopyPer - 1) / (kCopyNT * kCopyPer), 65535);
    return launch_chained(pages_copy_kernel<Unit>, dim3((unsigned)n, y), kCopyNT, 0, stream, p);
}

}  // namespace

size_t fork_workspace_bytes(int32_t n_seq, int32_t table_stride, int32_t n_pages) {
    const size_t rows = (size_t)n_seq * table_stride;
    return kWsHeader + ((size_t)n_pages + 63) / 64 * 256 + 4 * (2 * rows + 2 * (n_seq + rows / kPiece));
}

cudaError_t launch_pages_fork(int32_t n_seq, int32_t page_rows, const int32_t* parents, int64_t* lens, int32_t* table,
                              int32_t table_stride, int32_t* free_pages, int32_t* n_free, int32_t n_pages,
                              int32_t* copies, void* workspace, cudaStream_t stream) {
    ForkParams p{};
    p.n_seq = n_seq;
    while ((1 << p.shift) < page_rows) ++p.shift;
    p.stride = table_stride;
    p.n_pages = n_pages;
    p.parents = parents;
    p.lens = lens;
    p.table = table;
    p.free_pages = free_pages;
    p.n_free = n_free;
    p.copies = copies;
    char* ws = static_cast<char*>(workspace);
    p.err = reinterpret_cast<int32_t*>(ws);
    p.marks = reinterpret_cast<int32_t*>(ws + kWsHeader);
    p.rows = reinterpret_cast<int32_t*>(ws + kWsHeader + ((size_t)n_pages + 63) / 64 * 256);
    p.gone = p.rows + (size_t)n_seq * table_stride;
    p.counts = p.gone + (size_t)n_seq * table_stride;
    p.places = p.counts + n_seq + (size_t)n_seq * table_stride / kPiece;
    const cudaError_t e =
        cudaFuncSetAttribute(pages_fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(ForkShared));
    if (e != cudaSuccess) return e;
    return launch_chained(pages_fork_kernel, kCluster, kNT, sizeof(ForkShared), stream, p);
}

cudaError_t launch_pages_copy(int32_t n, const int32_t* copies, int32_t n_pages, int32_t n_pools,
                              const kvq_pool* pools, int32_t* err, cudaStream_t stream) {
    // pools whose pages start on 16 bytes, then the others
    for (int odd = 0; odd < 2; ++odd) {
        CopyParams p{};
        p.copies = copies;
        p.n_pages = n_pages;
        p.err = err;
        for (int32_t k = 0; k <= n_pools; ++k) {
            if (k < n_pools && (int)((((uintptr_t)pools[k].data | (uintptr_t)pools[k].page_bytes) & 15u) != 0) == odd)
                p.pool[p.n_pools++] = pools[k];
            if (p.n_pools == kMaxPools || (k == n_pools && p.n_pools > 0)) {
                const cudaError_t e = odd ? launch_copy<uint8_t>(p, n, stream) : launch_copy<uint4>(p, n, stream);
                if (e != cudaSuccess) return e;
                p.n_pools = 0;
            }
        }
    }
    return cudaSuccess;
}

}  // namespace kvq
