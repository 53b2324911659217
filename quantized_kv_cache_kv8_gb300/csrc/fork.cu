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
//   pass 1  marks[page] = kept        for the pages of sequences with children
//   pass 2  marks[page] = max(n - s)  for the other sequences s: the lowest is the page's owner
//   pass 3  new table rows, from the old ones, into the workspace; owned pages counted
//   pass 4  rows into the table, owned pages onto the stack in (sequence, page) order,
//           marks cleared, lengths and the free count written
//
// What bounds it: the latency of these dependent passes; the tables of a batch are a few
// hundred KB.  One cluster of 8 CTAs does it in one launch, with a cluster barrier
// between passes; CTA r owns a run of the (sequence, page) pairs.
#include "gqa.cuh"

#include <algorithm>
#include <cooperative_groups.h>

namespace kvq {
namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8, kNT = 1024, kWarps = kNT / 32;
constexpr int kMaxSeq = 4096;
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
};

struct ForkShared {
    int32_t first[kMaxSeq];     // a sequence's first child, n_seq without one
    int32_t pages[kMaxSeq + 1]; // pages of the sequences before it
    int32_t rank[kMaxSeq];      // of sequence i: copies before it, or -1
    int32_t part[kWarps];
    int32_t carry;
    int bad;
    int32_t count;              // owned pages of this CTA's pairs
    int32_t flag;               // this CTA met a page outside the pool
};

// Exclusive scan over the CTA of one value a thread; the total in *sum.
__device__ __forceinline__ int32_t scan(int32_t v, int32_t* part, int32_t* sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t t = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += t;
    }
    __syncthreads();
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    int32_t w = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t t = __shfl_up_sync(kFull, w, o);
        if (lane >= o) w += t;
    }
    *sum = __shfl_sync(kFull, w, 31);
    const int32_t before = __shfl_sync(kFull, w, max(warp - 1, 0));
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

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kNT) pages_fork_kernel(ForkParams p) {
    extern __shared__ __align__(16) unsigned char raw[];
    ForkShared& sm = *reinterpret_cast<ForkShared*>(raw);
    cg::cluster_group cluster = cg::this_cluster();
    launch_dependents();
    grid_dependency_wait();
    const int tid = threadIdx.x, cta = (int)cluster.block_rank(), n = p.n_seq;
    const int32_t P = 1 << p.shift;
    const int32_t n_free = *p.n_free;
    // the batch, by every CTA alike
    if (tid == 0) {
        sm.bad = n_free < 0 || n_free > p.n_pages;
        sm.carry = 0;
        sm.flag = 0;
    }
    for (int i = tid; i < n; i += kNT) sm.first[i] = n;
    __syncthreads();
    for (int i = tid; i < n; i += kNT) {
        const int32_t f = p.parents[i];
        const int64_t len = p.lens[i];
        if (f < -1 || f >= n || len < 0 || len > kMaxLen || ((len + P - 1) >> p.shift) > p.stride) sm.bad = 1;
        else if (f >= 0) atomicMin(&sm.first[f], i);
    }
    __syncthreads();
    const bool bad = sm.bad != 0;
    int32_t total = 0, copies = 0;   // pages of all sequences; copies
    if (!bad) {
        for (int k = 0; k < n; k += kNT) {
            const int i = k + tid;
            const int64_t len = i < n ? p.lens[i] : 0;
            int32_t sum;
            const int32_t at = scan((int32_t)((len + P - 1) >> p.shift), sm.part, &sum);
            if (i < n) sm.pages[i] = total + at;
            total += sum;
            const int32_t f = i < n ? p.parents[i] : -1;
            const bool copy = f >= 0 && sm.first[f] != i && (p.lens[f] & (P - 1)) != 0;
            const int32_t rank = scan(copy, sm.part, &sum);
            if (i < n) sm.rank[i] = copy ? copies + rank : -1;
            copies += sum;
        }
        if (tid == 0) sm.pages[n] = total;
    }
    __syncthreads();
    const int32_t status = bad ? KVQ_ERR_ARG : copies > n_free ? KVQ_ERR_WORKSPACE : KVQ_OK;
    // this CTA's pairs, a contiguous run
    const int32_t per = (int32_t)(((int64_t)total + kCluster - 1) / kCluster);
    const int32_t e0 = (int32_t)min((int64_t)cta * per, (int64_t)total), e1 = (int32_t)min((int64_t)e0 + per, (int64_t)total);
    if (status == KVQ_OK) {
        bool wrong = false;
        for (int32_t e = e0 + tid; e < e1; e += kNT) {
            const int s = find_last(sm.pages, n, e);
            const int32_t id = p.table[(int64_t)s * p.stride + (e - sm.pages[s])];
            if (id < 0 || id >= p.n_pages) wrong = true;
            else if (sm.first[s] < n) p.marks[id] = kKept;
        }
        // the pages that copies take
        for (int32_t i = cta * kNT + tid; i < copies; i += kCluster * kNT) {
            const int32_t id = p.free_pages[n_free - 1 - i];
            if (id < 0 || id >= p.n_pages) wrong = true;
        }
        if (wrong) sm.flag = 1;
    }
    __threadfence();
    cluster.sync();
    bool broken = status != KVQ_OK;
    for (int r = 0; r < kCluster; ++r) broken |= *cluster.map_shared_rank(&sm.flag, r) != 0;
    int32_t owned = 0;
    if (!broken) {
        for (int32_t e = e0 + tid; e < e1; e += kNT) {
            const int s = find_last(sm.pages, n, e);
            if (sm.first[s] < n) continue;
            int32_t* m = p.marks + p.table[(int64_t)s * p.stride + (e - sm.pages[s])];
            if (__ldcg(m) != kKept) atomicMax(m, n - s);
        }
        __threadfence();
    }
    cluster.sync();
    // a pair owns its page where its sequence is the lowest of the holders; a run's pairs are
    // dealt to the threads in consecutive pieces, so that ranks follow their order
    const int32_t piece = (e1 - e0 + kNT - 1) / kNT;
    const int32_t t0 = min(e0 + tid * piece, e1), t1 = min(t0 + piece, e1);
    if (!broken) {
        if (t0 < t1) {
            int s = find_last(sm.pages, n, t0);
            for (int32_t e = t0; e < t1; ++e) {
                while (e >= sm.pages[s + 1]) ++s;
                if (sm.first[s] < n) continue;
                owned += __ldcg(p.marks + p.table[(int64_t)s * p.stride + (e - sm.pages[s])]) == n - s;
            }
        }
        // new rows, column by column of this CTA's share
        for (int i = cta; i < n; i += kCluster) {
            const int32_t f = p.parents[i];
            if (f < 0) continue;
            const int32_t pages = sm.pages[f + 1] - sm.pages[f];
            for (int32_t w = tid; w < pages; w += kNT) {
                int32_t id = p.table[(int64_t)f * p.stride + w];
                if (w == pages - 1 && sm.rank[i] >= 0) {
                    const int32_t to = p.free_pages[n_free - 1 - sm.rank[i]];
                    p.copies[2 * i] = id;
                    p.copies[2 * i + 1] = to;
                    id = to;
                }
                p.rows[(int64_t)i * p.stride + w] = id;
            }
        }
    }
    int32_t sum;
    int32_t rank = scan(owned, sm.part, &sum);
    if (tid == 0) sm.count = sum;
    __threadfence();
    cluster.sync();
    int32_t freed = 0;
    for (int r = 0; r < kCluster; ++r) {
        const int32_t c = *cluster.map_shared_rank(&sm.count, r);
        if (r < cta) rank += c;
        freed += c;
    }
    // a page listed twice by one sequence could be let go twice: the stack has room for the pool
    const bool full = (int64_t)n_free - copies + freed > p.n_pages;
    if (!broken && !full) {
        if (owned > 0) {
            int s = find_last(sm.pages, n, t0);
            for (int32_t e = t0; e < t1; ++e) {
                while (e >= sm.pages[s + 1]) ++s;
                if (sm.first[s] < n) continue;
                const int32_t id = p.table[(int64_t)s * p.stride + (e - sm.pages[s])];
                if (__ldcg(p.marks + id) == n - s) {
                    p.free_pages[n_free - copies + freed - 1 - rank] = id;
                    ++rank;
                }
            }
        }
    }
    __threadfence();
    cluster.sync();   // marks and the old table are read
    if (status == KVQ_OK)
        for (int32_t e = e0 + tid; e < e1; e += kNT) {
            const int s = find_last(sm.pages, n, e);
            const int32_t id = p.table[(int64_t)s * p.stride + (e - sm.pages[s])];
            if (id >= 0 && id < p.n_pages) p.marks[id] = 0;
        }
    if (broken || full) {
        if (cta == 0) {
            if (tid == 0 && p.err) atomicCAS(p.err, 0, status != KVQ_OK ? status : (int32_t)KVQ_ERR_ARG);
        }
        for (int i = cta * kNT + tid; i < n; i += kCluster * kNT) p.copies[2 * i] = p.copies[2 * i + 1] = -1;
        cluster.sync();
        return;
    }
    // lengths are read by all before one CTA writes them; so is the old table
    int64_t len[(kMaxSeq + kNT - 1) / kNT];
    if (cta == 0)
        for (int k = 0, i = tid; i < n; i += kNT, ++k) {
            const int32_t f = p.parents[i];
            len[k] = f >= 0 ? p.lens[f] : 0;
        }
    cluster.sync();
    if (cta == 0) {
        for (int k = 0, i = tid; i < n; i += kNT, ++k) p.lens[i] = len[k];
        if (tid == 0) *p.n_free = n_free - copies + freed;
    }
    for (int i = cta; i < n; i += kCluster) {
        const int32_t f = p.parents[i];
        if (tid == 0 && sm.rank[i] < 0) p.copies[2 * i] = p.copies[2 * i + 1] = -1;
        if (f < 0) continue;
        const int32_t pages = sm.pages[f + 1] - sm.pages[f];
        for (int32_t w = tid; w < pages; w += kNT)
            p.table[(int64_t)i * p.stride + w] = p.rows[(int64_t)i * p.stride + w];
    }
}

constexpr int kCopyNT = 256, kMaxPools = 128;
constexpr int64_t kPiece = 16384;   // bytes of a page that a CTA copies

struct CopyParams {
    const int32_t* copies;
    int32_t n_pages, n_pools;
    int32_t* err;
    kvq_pool pool[kMaxPools];
    int32_t piece0[kMaxPools + 1];   // pieces of the pools before it
};

// One piece of one page of one pool a CTA.  What bounds it: memory.
__global__ void __launch_bounds__(kCopyNT) pages_copy_kernel(const __grid_constant__ CopyParams p) {
    launch_dependents();
    grid_dependency_wait();
    const int i = blockIdx.x;
    const int32_t from = p.copies[2 * i], to = p.copies[2 * i + 1];
    if (from < 0 || to < 0) return;
    if (from >= p.n_pages || to >= p.n_pages) {
        if (threadIdx.x == 0 && p.err) atomicCAS(p.err, 0, (int32_t)KVQ_ERR_ARG);
        return;
    }
    for (int32_t y = blockIdx.y; y < p.piece0[p.n_pools]; y += gridDim.y) {
        const int k = find_last(p.piece0, p.n_pools, y);
        const int64_t bytes = p.pool[k].page_bytes, b0 = (y - p.piece0[k]) * kPiece, b1 = min(b0 + kPiece, bytes);
        char* base = static_cast<char*>(p.pool[k].data);
        const char* src = base + from * bytes;
        char* dst = base + to * bytes;
        if ((((uintptr_t)base | (uintptr_t)bytes) & 15u) == 0) {
            uint4 v[kPiece / 16 / kCopyNT];
#pragma unroll
            for (int u = 0; u < kPiece / 16 / kCopyNT; ++u) {
                const int64_t at = b0 + 16 * (u * kCopyNT + (int)threadIdx.x);
                if (at < b1) v[u] = *reinterpret_cast<const uint4*>(src + at);
            }
#pragma unroll
            for (int u = 0; u < kPiece / 16 / kCopyNT; ++u) {
                const int64_t at = b0 + 16 * (u * kCopyNT + (int)threadIdx.x);
                if (at < b1) *reinterpret_cast<uint4*>(dst + at) = v[u];
            }
        } else {
            for (int64_t at = b0 + threadIdx.x; at < b1; at += kCopyNT) dst[at] = src[at];
        }
    }
}

}  // namespace

size_t fork_workspace_bytes(int32_t n_seq, int32_t table_stride, int32_t n_pages) {
    return kWsHeader + ((size_t)n_pages + 63) / 64 * 256 + (size_t)n_seq * table_stride * 4;
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
    const cudaError_t e =
        cudaFuncSetAttribute(pages_fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(ForkShared));
    if (e != cudaSuccess) return e;
    return launch_chained(pages_fork_kernel, kCluster, kNT, sizeof(ForkShared), stream, p);
}

cudaError_t launch_pages_copy(int32_t n, const int32_t* copies, int32_t n_pages, int32_t n_pools,
                              const kvq_pool* pools, int32_t* err, cudaStream_t stream) {
    for (int32_t k0 = 0; k0 < n_pools; k0 += kMaxPools) {
        CopyParams p{};
        p.copies = copies;
        p.n_pages = n_pages;
        p.n_pools = std::min(kMaxPools, n_pools - k0);
        p.err = err;
        int64_t pieces = 0;
        for (int32_t k = 0; k < p.n_pools; ++k) {
            p.pool[k] = pools[k0 + k];
            p.piece0[k] = (int32_t)pieces;
            pieces += (p.pool[k].page_bytes + kPiece - 1) / kPiece;
            if (pieces > 0x7fffffff) return cudaErrorInvalidConfiguration;
        }
        p.piece0[p.n_pools] = (int32_t)pieces;
        if (pieces == 0) continue;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)n, (unsigned)std::min<int64_t>(pieces, 65535));
        cfg.blockDim = dim3(kCopyNT);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, pages_copy_kernel, p);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace kvq
