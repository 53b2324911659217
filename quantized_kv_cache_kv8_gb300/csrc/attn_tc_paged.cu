// attn_tc_paged.cu -- tensor-core attention of new tokens over paged KV8 or TQ4
// rows, bf16 queries, on pairs of CTAs.
//
// A pair (a cluster of two CTAs on neighbouring SMs) walks over segments
// (paged_common.cuh): 128 query vectors -- consecutive (token, head) pairs of
// one sequence, whatever the head count, 64 to a CTA -- against a run of 128-row
// steps.  Both products run as cta_group::2 MMAs with M = 128, issued by the
// first CTA:
//   S = Q C^T   N = 128 rows, K = 576 dims; latent and rope dims into an
//               accumulator each, as each has its own row scale
//   O += P C    N = 256 dims, twice, K = 128 rows
// The pair shares the B operands: a CTA supplies 64 of the step's rows (all
// dims) to the scores and 256 of the latent dims (all rows) to the context.
// That decides the layout.  One CTA alone, with rows on M and 64 vectors on N,
// reads 6 KB of operands for each 32 cycles of products, where shared memory
// delivers 128 B a cycle (48 cycles; 575 KB a step with the decoded stores, 4.5k
// cycles); here the scores read 4 KB in 32 cycles and the context 6 KB in 64 (243 KB
// and 1.9k with KV8's scores in fp8, 540 KB and 4.2k with TQ4's in two halves of f16).  More
// vectors a CTA do not fit: 64 x 512 f32 of context are half of a CTA's tensor memory.
//
// Operands.  KV8: the scores run as fp8 MMAs on the codes themselves: TMA puts
// them into swizzled shared memory page by page, no warp touches them, and they
// take half the space of f16 (so a step's latent dims are loaded while the step
// before is in use).  A bf16 query vector times a power of two of its own is
// q1 + q2 in e4m3, the upper and the lower 4 of its 8 significant bits (exact for
// elements over 2^-9 of the largest, off by at most 2^-17 of the largest below),
// so each K step runs twice, with q1 and q2, in the time of one f16 step.  The
// context needs weights with more range than fp8 has: its rows are decoded to f16
// (e4m3 codes exactly).
// TQ4: levels are no fp8 values; both operands are decoded to f16 (the 16 levels
// times kGamma within 9.3e-5), and the rotated query is q1 + q2 in f16, value and
// residual, 22 bits (one f16 alone moves outputs by up to 3e-3 of the largest).  The
// second half takes the space of the score rows, so score and context rows of a step go
// through two slots of 32 KB in five fills: three times three chunks of the score rows, then
// context rows 0-63 and 64-127.  (With the rope dims in a fill of their own, the next fill
// waits for the products of the one before it: 256 tokens on 16,384 rows 2.01 ms.  Four
// warps for the scores and four for the context, slots of 16 KB each: 1.99.)
//
// Roles (a CTA): 8 softmax warps, 8 decode warps, one issuing warp (in the first
// CTA; the second's passes on that its codes have arrived), one that announces
// segments, one that fetches row scales, one that loads codes by TMA; registers
// move to the warps that need them (Regs).  The decode warps store the context rows of
// step t once the context of step t-1 is complete (KV8), or each fill once the products of
// the fill before the last are (TQ4); the scores of t+1 are issued before the
// context of t.  So the tensor pipe alternates between the two while the other
// operand is being stored and while the softmax of the step runs:
//   tensor   S(t)   O(t-1)    S(t+1)    O(t)
//   decode          K(t+1)    V(t)      K(t+2)  ...
//   softmax         ---- P(t) ----      -- P(t+1) --
// Accumulators: O 256 columns, S two buffers of 64 + 64.
//
// Softmax, per query vector (a thread has one and a quarter of the rows), in log2
// units: m is a lagged running maximum of the scores, p = 2^(z - m) enters the
// row sum in f32, and the context takes the f16 weight w = p s_L E,
// E = 2^(m - R - 2) with R the largest z + log2 s_L of the steps that set the
// references, so that weights are relative to the largest p s_L and rows of
// small latent scale keep f16 precision where they matter.  A step in which w might
// pass 2^15.75, by its largest z - m and its largest s_L, goes down the exact path: row
// maxima, new m, R and E, O rescaled in tensor memory.  (A bound of its own for each,
// 2^14 and 3.5, sent more steps there: mixed batch of 24 sequences 212 us, 206 with the
// one for both; 235 with 2^10.)  Rows that a vector does not see get
// z = -inf; a vector that has seen no row has m = -inf and E = 0.
//
// Weights under 2^-14 lose bits, up to 2^-25 a row: nothing beside one large weight, but
// 131,072 rows 20 binades below the first lost a third of their sum, 3% of the output.  So
// each thread keeps the sum of its weights and that bound of what it lost (32 rows a
// step).  Where the loss may pass 2^-11 of the sum, the step takes the exact path and R
// comes down to its largest z + log2 s_L, by 2^24 at most; each fall after that waits for a
// sixteenth of it (2^24 steps, then).  A vector's largest weight is one thread's, so the
// least of its four sums is at most a third of all its weights, and less than 2^-10 of them
// is lost before the first fall, beside the 2^-11 of its own by which any weight is rounded.
// (A larger E has fewer falls and more rises: mixed batch of 24 sequences 206 us; 213 with
// 2^(m - R - 3), 211 with 2^(m - R).)
//
// The products round their f32 sums towards zero: what the 65,536 MMAs of a million rows
// add to one accumulator came out 0.3% small, and 3% off where the first row outweighs the
// rest.  So the sums run in two levels: every kFold steps (32,768 rows) the softmax warps
// add O, and the row sum, to totals, O's in the walker's second slot of the workspace (free
// until its last segment ends), and the next product starts from zero (1 to 2% of a long
// walk).
//
// What bounds it.  KV8, many rows a tile: the softmax warps, some 3,450 cycles a step (scores
// 1,350, vote 290, exponentials 600, weights 500, the rest hand-overs) for 2,200 of
// products: 512 tokens on 32,768 rows x 128 heads 3.2 ms, 1,470 TFLOP/s; 32 sequences of
// 1,024 to 131,072 rows 360 us.  TQ4: the hand-over of the fills, 7,700 a step for 3,350
// of products; no pipe is full (integer 46%, tensor 44%, issue slots 41%; 256 tokens on
// 16,384 rows 1.78 ms, 660 TFLOP/s).  Short tiles: rotation of queries and
// outputs (TQ4, 777 tokens without rows before 319 us), and the start (6k cycles), the
// queries (8k) and the partial results (6k) of a decode step (8 x 4096 rows 27.1 us).
#include "tc_common.cuh"
#include "paged_common.cuh"

#include <cuda.h>
#include <math.h>

namespace kvq {
namespace {
using namespace tc;

constexpr int kRows = PagedTensor::kN;       // rows a step
constexpr int kVecs = PagedTensor::kM;       // query vectors of the pair
constexpr int kHalf = 64;                    // query vectors, and score rows, of a CTA
static_assert(kRows == 2 * kHalf && kVecs == 2 * kHalf, "pair layout");
constexpr int kSoftWarps = 8, kDecWarps = 8;
constexpr int kSoft = 32 * kSoftWarps, kDec = 32 * kDecWarps;
constexpr int kIssueWarp = kSoftWarps + kDecWarps, kWalkWarp = kIssueWarp + 1, kScaleWarp = kIssueWarp + 2,
              kLoadWarp = kIssueWarp + 3;
constexpr int kThreads = kSoft + kDec + 128;   // five warpgroups
// Registers a thread after the split.  KV8: the decode warps hold half the codes
// (none of the score rows), and the softmax keeps a step's latent scales between scores
// and weights instead of reading them twice (32 sequences of 1,024 to 131,072 rows 360 us,
// 368 with 112 and 96 registers).
template <bool TQ4>
struct Regs {
    static constexpr int kLaunch = 96, kSoftmax = TQ4 ? 88 : 120, kDecode = TQ4 ? 120 : 88, kRest = 64;
    static_assert(kSoft * kSoftmax + kDec * kDecode + 128 * kRest <= kThreads * kLaunch, "register split");
};
// To N from the launch's count, by a whole warpgroup (N = FROM is written too: the
// compiler allots a branch the registers that it names).
template <int N, int FROM>
__device__ __forceinline__ void set_registers() {
    if constexpr (N > FROM) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
constexpr int kCols = 32;                    // rows of a step that a softmax thread has
constexpr int kChunks = 9, kRope = 8;        // TQ4: 64-dim f16 chunks of a row, 8 latent, 1 rope
constexpr uint32_t kChunkBytes = kHalf * 128;   // 64 rows (or vectors) x 64 f16
constexpr uint32_t kVChunkBytes = kRows * 128;  // 128 rows x 64 f16
// KV8, the same nine places of 8 KB: queries q1 of 4 x 128 dims, q2 likewise, rope
// (q1 in the lower 64 bytes of a row, q2 in the upper); codes of 4 x 128 dims of two
// steps, and the row's last 128 bytes (the rope dims are the upper 64).
// TQ4: q1, then q2 in the nine places after it; the slots where KV8 has its context rows.
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = kOffQ + kChunks * kChunkBytes;
constexpr uint32_t kOffV = kOffK + kChunks * kChunkBytes;   // 4 chunks: dims 256 j + 128 rank + 64 i
constexpr uint32_t kOffSlot = kOffV, kSlotBytes = 4 * kChunkBytes;   // TQ4
static_assert(2 * kSlotBytes <= 4 * kVChunkBytes, "slots");
constexpr uint32_t kOffP = kOffV + 4 * kVChunkBytes;        // weights: 2 chunks of 64 rows
constexpr uint32_t kOffScale = kOffP + 2 * kChunkBytes;     // s_L, then s_R, of two steps' rows
constexpr uint32_t kScaleBytes = kRows * 8;
constexpr uint32_t kOffCz = kOffScale + 2 * kScaleBytes;    // score scale of a vector, two segments
constexpr uint32_t kOffBar = kOffCz + 2 * kHalf * 4;
constexpr uint32_t kOffMax = kOffBar + 26 * 8;              // log2 of the largest s_L of two steps
constexpr uint32_t kOffLevels = kOffMax + 16;
constexpr uint32_t kOffMisc = kOffLevels + 16;              // abort flag, TMEM base
constexpr uint32_t kOffWork = kOffMisc + 16;                // two segments, announced one ahead
constexpr uint32_t kSmemUsed = kOffWork + 2 * 72;
constexpr uint32_t kOffPart = kOffScale;                    // scan of the work split, before the steps
static_assert(kWalkScratch<kThreads> * 8 <= 2 * kScaleBytes, "scan scratch");
static_assert(kOffK % 1024 == 0 && kOffV % 1024 == 0 && kOffP % 1024 == 0 && kOffWork % 8 == 0, "alignment");
static_assert(kSmemUsed <= 232448, "shared memory budget");
static_assert(32 * kMlaDV * 4 <= 4 * kVChunkBytes, "output stage");

constexpr uint32_t kColO = 0, kColS = 256, kTmemCols = 512;

// mbarriers.  In the first CTA, arrivals from both: slots stored (TQ4), context rows
// stored (KV8: rows 0-63, 64-127), weights written.  In
// each CTA: scores complete and their row scales stored (by buffer; commits reach
// both CTAs), context complete (by row half), segment announced, segment done
// with, queries stored, output written, row scales read,
// every product complete, and one that nothing arrives on (the testing hook).
enum {
    kBarK0 = 0, kBarV0 = 2, kBarP = 4, kBarScore0 = 5, kBarCtx0 = 7, kBarWork0 = 9, kBarWorkFree0 = 11, kBarQ0 = 13, kBarOut = 15,
    kBarDone = 16, kBarNever = 17, kBarScaleFree0 = 18,
    // KV8: latent codes of a step (two buffers) and its rope codes have arrived
    // here; in the first CTA, that they have arrived in the second
    kBarLat0 = 20, kBarRope = 22, kBarPeerLat0 = 23, kBarPeerRope = 25, kNumBars = 26,
    kBarQFirst = kBarK0,  // KV8, in the first CTA: queries stored in both
    // TQ4, by slot: stored in both CTAs (in the first), its products complete (in each)
    kBarFull0 = kBarK0, kBarFree0 = kBarLat0
};
// Scores, announcements, queries and scales have two barriers each, used in turn:
// their next but one event waits for whoever waits for this one, the next does not.

constexpr float kLogWmax = 15.75f, kHeadroom = 2.0f, kLogEmax = 120.0f, kLogMax = 100.0f;
constexpr int kFold = 256;   // steps that one accumulator sums
constexpr float kLossStep = 0x1p-20f, kLossShare = 0x1p-11f, kMaxDrop = 24.0f;
static_assert(kCols == 32, "a thread's rows a step, 2^-25 each");
// levels times this round to f16 within 9.3e-5 (unscaled: 3.2e-4); divided out in f32
constexpr float kGamma = 1.3338516f;
constexpr uint32_t kIdescScore = idesc_f16(kVecs, kRows, false, false);   // e4m3 x e4m3 has the same bits
constexpr uint32_t kIdescCtx = idesc_f16(kVecs, 256, false, true);

// A segment as the roles use it; steps = 0 ends the walk.
struct Work {
    int32_t steps, b, rows;
    int32_t first, end, seen0;   // first row; rows that some vector sees; rows that the first one sees
    int64_t row0, tok0, base, slot;
    int32_t parts, pad;
};
static_assert(sizeof(Work) <= 72, "segment record");

// ---- pair-wide barriers and MMAs ----------------------------------------------
__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
// The same for waits that last for many steps: half a microsecond between polls.
__device__ __forceinline__ bool idle_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, long long limit) {
    for (long long i = 0; i < limit; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if (*abort_flag) return false;
        __nanosleep(500);
    }
    *abort_flag = 1;
    return false;
}
// A warp's bounded wait.  The abort flag is read between polls only: a shared
// load takes some 200 cycles next to the operand reads of the products.
__device__ __forceinline__ bool try_once(uint32_t a, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(a), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, long long limit) {
    const uint32_t a = smem_u32(bar);
    if (__all_sync(kFull, try_once(a, parity))) return true;
    bool ok = false;
    for (long long i = 0; i < limit; ++i) {
        if (__all_sync(kFull, try_once(a, parity))) {
            ok = true;
            break;
        }
        if ((i & 63) == 63 && __any_sync(kFull, *abort_flag != 0)) break;
    }
    if (!ok) *abort_flag = 1;
    return ok;
}

// One arrival of a warp on a barrier of its own CTA, or of the first CTA.  What
// an arrival announces is this CTA's shared memory, read by this SM's tensor
// core: the async-proxy fence before it has put the stores there, so the arrival
// releases at CTA scope only (a release at cluster scope waits for every
// outstanding access of the warp, 1,000 cycles each time, 2.4 of the 4.1 us of a step).
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}
__device__ __forceinline__ void warp_arrive_first(uint64_t* bar, int lane) {
    __syncwarp();
    if (lane == 0) {
        uint32_t a;
        asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(bar)));
        asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(a) : "memory");
    }
}
// One MMA, or one commit, of a whole warp in step: the warp computes the
// descriptors together (in uniform registers) and one elected lane, always the
// same, issues.  A lone lane in a branch of its own spends about 115 cycles an
// MMA on moving its operands, more than the MMA takes.
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
        " @q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void pair_mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
        " @q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
    asm volatile(
        "{\n .reg .pred q;\n .reg .b16 m;\n mov.b16 m, 3;\n elect.sync _|q, 0xffffffff;\n"
        " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n}\n" ::"r"(
            smem_u32(bar))
        : "memory");
}

// A barrier of the four softmax warps that share 32 vectors (group 0 or 1), and the
// same with a vote.  The groups' references are their own: they part and meet at the
// segment's end only.
__device__ __forceinline__ void group_sync(int group) {
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(2 + group) : "memory");
}
__device__ __forceinline__ bool group_any(int group, bool v) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(2 + group)
        : "memory");
    return r != 0;
}

// ---- loads (KV8) --------------------------------------------------------------
__device__ __forceinline__ void expect_bytes(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
// A box of pool rows [y, y + box) x bytes [x, x + 128), x a multiple of 16.
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* map, int32_t x, int32_t y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y)
        : "memory");
}

// ---- decode -------------------------------------------------------------------
// KV8: 16 codes, a quarter of a row's 64-dim chunk, 32 bytes of f16 in two 16-byte
// stores.  A warp reads 256 dims of two rows; the 8 lanes that a store serves at a time
// have one chunk of both rows, whose swizzle phases differ in the low bit: 8 different
// 16-byte units.

// The f16 levels of codes 8-15 as byte planes, four levels a word; those of codes
// 7-0 are their negatives.
struct Planes {
    uint32_t lo[2], hi[2];
};
constexpr bool levels_mirror() {
    for (int k = 0; k < 8; ++k)
        if (kTq4LevelBits[7 - k] != (kTq4LevelBits[8 + k] ^ 0x80000000u)) return false;
    return true;
}
static_assert(levels_mirror(), "decode takes the lower levels from the upper ones");
// e4m3: a NaN code becomes the lowest value, for a row counts, weight 0, in the
// context of the vectors that do not see it too; those that do get their NaN from
// its score.
__device__ __forceinline__ void store_codes(unsigned char* chunk, const uint4& c, int row, int q) {
    const uint32_t in[4] = {c.x, c.y, c.z, c.w};
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) e4m3x4_to_half2x2(in[i], w[2 * i], w[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("max.f16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(0xdf00df00u));   // -448
    *reinterpret_cast<uint4*>(chunk + sw128(row, 32 * q)) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(chunk + sw128(row, 32 * q + 16)) = make_uint4(w[4], w[5], w[6], w[7]);
}
// Nibble codes by byte permutes over the low and the high bytes of the levels: the
// low 3 bits of a code (their complement below 8) pick the level, bit 3 its sign.
// Eight of them, one word, fill a 16-byte unit.
__device__ __forceinline__ void store_levels(unsigned char* chunk, uint32_t codes, int row, int unit, const Planes& t) {
    const uint32_t neg = ~codes & 0x88888888u, even = neg << 4;   // signs in bit 7 of a byte: odd codes, even codes
    // 7/8 of it, 7 in each code below 8, by a high product: the integer pipe is the
    // busiest one (256 tokens on 16,384 rows 1.78 ms, 1.80 with a shift and a difference)
    const uint32_t sel = (codes & 0x77777777u) ^ __umulhi(neg, 0xe0000000u);
    uint32_t w[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t s = h ? sel >> 16 : sel;
        const uint32_t lo = __byte_perm(t.lo[0], t.lo[1], s);
        const uint32_t hi = __byte_perm(t.hi[0], t.hi[1], s) | (__byte_perm(even, neg, h ? 0x7362u : 0x5140u) & 0x80808080u);
        w[2 * h] = __byte_perm(lo, hi, 0x5140u);
        w[2 * h + 1] = __byte_perm(lo, hi, 0x7362u);
    }
    *reinterpret_cast<uint4*>(chunk + sw128(row, 16 * unit)) = make_uint4(w[0], w[1], w[2], w[3]);
}

// ---- queries ------------------------------------------------------------------
// Prologue and epilogue run once a segment, with few warps: what counts is the
// chain of each warp, so a warp takes four vectors at once, 8 lanes each (l = lane % 8),
// and no transform crosses lanes where shared memory can turn the data instead.

// The unscaled transform, stage by stage.
__device__ __forceinline__ void butterfly(F2& a, F2& b) {
    const F2 s = add2(a, b);
    b = fma2(b, f2(-1.0f, -1.0f), a);
    a = s;
}
// Within the units, over the first index of x.
template <int N>
__device__ __forceinline__ void transform_in(F2 (&x)[N][2]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float2 e = unpack(x[i][k]);
            x[i][k] = f2(e.x + e.y, e.x - e.y);
        }
        butterfly(x[i][0], x[i][1]);
    }
}
template <int N, int K>
__device__ __forceinline__ void transform_over(F2 (&x)[N][K]) {
#pragma unroll
    for (int h = 1; h < N; h <<= 1)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if ((i & h) == 0)
#pragma unroll
                for (int k = 0; k < K; ++k) butterfly(x[i][k], x[i + h][k]);
}
// Over the 8 lanes of a vector.
template <int N>
__device__ __forceinline__ void transform_lanes(F2 (&x)[N][2], int lane) {
#pragma unroll
    for (int h = 1; h < 8; h <<= 1) {
        const float sign = (lane & h) ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float2 e = unpack(x[i][k]);
                x[i][k] = fma2(f2(sign, sign), x[i][k], f2(__shfl_xor_sync(kFull, e.x, h), __shfl_xor_sync(kFull, e.y, h)));
            }
    }
}
// Flips the elements of v whose sign bit is set in words w of a block.
template <int N>
__device__ __forceinline__ void apply_signs(float (&v)[N][4], const uint64_t* w, int l) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t half = (uint32_t)(w[i >> 1] >> (32 * (i & 1)));   // 32 signs: units 8 i .. 8 i + 7
        const uint32_t bits = half >> (4 * l);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[i][k] = __int_as_float(__float_as_int(v[i][k]) ^ (int)((bits >> k) << 31));
    }
}

// What both loaders do with a vector's largest magnitude (as bits: a NaN counts above
// an infinity): 2^shift puts it into [2^(TOP-1), 2^TOP); |shift| <= 114 keeps that and
// its inverse normal numbers.  A vector with a NaN or an infinity becomes NaN
// throughout (e4m3 would saturate the infinity).  Returns 2^shift; *undo gets 2^-shift.
template <int TOP>
__device__ __forceinline__ float vector_scale(uint32_t top, float* undo) {
#pragma unroll
    for (int h = 1; h < 8; h <<= 1) top = max(top, __shfl_xor_sync(kFull, top, h));
    const bool finite = top < 0x7f800000u;
    const int shift = top == 0u || !finite ? 0 : min(114, TOP + 126 - max((int)(top >> 23), 1));
    *undo = __uint_as_float((uint32_t)(127 - shift) << 23);
    return finite ? __uint_as_float((uint32_t)(127 + shift) << 23) : __uint_as_float(0x7fffffffu);
}

// This CTA's 64 vectors, 8 a decode warp, under a power of two of their own; sCz gets
// what undoes it in the score.  KV8: to a sum of two e4m3 values.
__device__ __forceinline__ void load_queries(const PagedParams& p, int64_t row0, int rows, unsigned char* sQ,
                                             float* sCz, int warp, int lane) {
    constexpr int kUnits = 18;   // units of a lane: 16 latent, 2 rope
    const int l = lane & 7;
    const int r0 = (kHalf / kDecWarps) * warp + (lane >> 3);
    const uint2* src = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.q) + (row0 + r0) * kMlaD) + l;
    uint2 raw[kUnits], ahead[kUnits];
    auto fetch = [&](int g, uint2 (&raw)[kUnits]) {
        const bool ok = r0 + 4 * g < rows;
#pragma unroll
        for (int i = 0; i < kUnits; ++i)
            raw[i] = ok ? src[g * kMlaD + 8 * i] : make_uint2(0u, 0u);   // 4 vectors on: 4 * 144 units
    };
    fetch(0, raw);
    fetch(1, ahead);
#pragma unroll 1
    for (int g = 0; g < 2; ++g) {
        const int r = r0 + 4 * g;
        uint32_t both = 0u;
#pragma unroll
        for (int i = 0; i < kUnits; ++i)
            both = __vmaxu2(both, __vmaxu2(raw[i].x & 0x7fff7fffu, raw[i].y & 0x7fff7fffu));
        float undo;
        const float scale = vector_scale<8>(max(both << 16, both & 0xffff0000u), &undo);
        if (l == 0) sCz[r] = p.sm_scale * kLog2e * undo;
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int u = l + 8 * (i < 16 ? i : i - 16);   // unit of the latent or of the rope dims
            // 8 significant bits under 256: exact in f16, as is what q1 leaves
            uint32_t c1[2], c2[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t w = h ? raw[i].y : raw[i].x;
                const __half2 x = __floats2half2_rn(__uint_as_float(w << 16) * scale, __uint_as_float(w & 0xffff0000u) * scale);
                const __nv_fp8x2_storage_t f1 = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE, __NV_E4M3);
                const __half2 rest = __hsub2(x, __half2(__nv_cvt_fp8x2_to_halfraw2(f1, __NV_E4M3)));
                c1[h] = f1;
                c2[h] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(rest), __NV_SATFINITE, __NV_E4M3);
            }
            unsigned char* c = sQ + (i < 16 ? i >> 2 : kRope) * kChunkBytes;
            const int byte = i < 16 ? 4 * (u & 31) : 4 * u;
            *reinterpret_cast<uint32_t*>(c + sw128(r, byte)) = c1[0] | c1[1] << 16;
            *reinterpret_cast<uint32_t*>(i < 16 ? c + 4 * kChunkBytes + sw128(r, byte) : c + sw128(r, 64 + byte)) =
                c2[0] | c2[1] << 16;
        }
#pragma unroll
        for (int i = 0; i < kUnits; ++i) raw[i] = ahead[i];
    }
}

// TQ4: rotated, to q1 + q2 in f16.  A lane begins with dims 8 (l + 8 j) .. + 7 of its
// vector, six of the nine stages in its registers; 8 KB of shared memory turn that into
// the 64 dims of chunk l for the other three (shuffles for them take longer than the rest
// of the transform).  The warp's eight vectors are one 1 KB atom of each chunk, its own: the
// first four are turned, and written, while the last four rows of 16 atoms hold the turn,
// the last four come to lie where they were turned.
__device__ __forceinline__ uint32_t to_half2(F2 x) {
    const float2 e = unpack(x);
    const __half2 h = __floats2half2_rn(e.x, e.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void rotate_queries(const PagedParams& p, int64_t row0, int rows, unsigned char* sQ,
                                               float* sCz, int warp, int lane) {
    const int l = lane & 7, v4 = lane >> 3;
    const int r0 = (kHalf / kDecWarps) * warp + v4;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + (row0 + r0) * kMlaD) + l;
    static_assert(kHalf / kDecWarps == 8, "a warp has an atom of each chunk");
    // a vector's 2 KB: the half atoms of four latent chunks (of q1: vectors 0, 1; of q2: 2, 3)
    unsigned char* own = sQ + (v4 < 2 ? 4 * v4 : 4 * v4 + kChunks - 8) * kChunkBytes + 1024 * warp + 512;
    // place of unit u (four dims): 8 lanes, 2 or 16 units apart, on different banks
    auto at = [own](int u) {
        const int x = u ^ ((u >> 3) & 7) ^ ((u >> 6) & 1);
        return reinterpret_cast<float4*>(own + (x >> 5) * kChunkBytes + 16 * (x & 31));
    };
    uint4 raw[9];
    auto fetch = [&](int g) {
        const bool ok = r0 + 4 * g < rows;
#pragma unroll
        for (int j = 0; j < 9; ++j) raw[j] = ok ? src[g * 4 * (kMlaD / 8) + 8 * j] : make_uint4(0u, 0u, 0u, 0u);
    };
    // two elements with their signs (the lowest two bits) applied
    auto pair = [](uint32_t w, uint32_t bits) {
        w ^= (bits & 1u) << 15 | (bits & 2u) << 30;
        return f2(w << 16, w & 0xffff0000u);
    };
    fetch(0);
#pragma unroll 1
    for (int g = 0; g < 2; ++g) {
        const int r = r0 + 4 * g;
        F2 x[16][2], rope[2][2];
#pragma unroll
        for (int j = 0; j < 9; ++j) {   // the rope block's word follows the latent block's 8
            const uint32_t bits = (uint32_t)(p.signs.w[j] >> (8 * l));
            F2 (&a)[2] = j < 8 ? x[j < 8 ? 2 * j : 0] : rope[0], (&b)[2] = j < 8 ? x[j < 8 ? 2 * j + 1 : 0] : rope[1];
            a[0] = pair(raw[j].x, bits);
            a[1] = pair(raw[j].y, bits >> 2);
            b[0] = pair(raw[j].z, bits >> 4);
            b[1] = pair(raw[j].w, bits >> 6);
        }
        if (g == 0) fetch(1);
        transform_in(x);
        transform_over(x);
        transform_in(rope);
        transform_over(rope);
        transform_lanes(rope, lane);
        __syncwarp();   // the group before has been read
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 a = unpack(x[i][0]), b = unpack(x[i][1]);
            *at(2 * (l + 8 * (i >> 1)) + (i & 1)) = make_float4(a.x, a.y, b.x, b.y);
        }
        __syncwarp();
        F2 y[8][4];   // dims 64 l + 8 m + 2 k, + 1
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 v = *at(2 * (m + 8 * l) + h);
                y[m][2 * h] = f2(v.x, v.y);
                y[m][2 * h + 1] = f2(v.z, v.w);
            }
        transform_over(y);
        uint32_t top = 0u;
        auto scaled = [&](F2 v, float kn) {
            v = mul2(v, f2(kn, kn));
            const float2 e = unpack(v);
            top = max(top, max(__float_as_uint(e.x) & 0x7fffffffu, __float_as_uint(e.y) & 0x7fffffffu));
            return v;
        };
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int m = 0; m < 8; ++m) y[m][k] = scaled(y[m][k], p.kn[0]);
            rope[k >> 1][k & 1] = scaled(rope[k >> 1][k & 1], p.kn[1]);
        }
        float undo;
        const float scale = vector_scale<14>(top, &undo);
        if (l == 0) sCz[r] = p.sm_scale * kLog2e * undo * (1.0f / kGamma);
        const F2 s2 = f2(scale, scale);
        __syncwarp();   // the turn has been read: the last four rows' places too
        auto store = [&](int chunk, int byte, F2 a, F2 b, F2 c, F2 d) {
            const F2 x[4] = {mul2(a, s2), mul2(b, s2), mul2(c, s2), mul2(d, s2)};
            uint32_t q1[4], q2[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 e = unpack(x[i]);
                const __half2 h = __floats2half2_rn(e.x, e.y);
                const float2 back = __half22float2(h);
                q1[i] = *reinterpret_cast<const uint32_t*>(&h);
                q2[i] = to_half2(f2(e.x - back.x, e.y - back.y));   // the difference is exact
            }
            unsigned char* to = sQ + chunk * kChunkBytes + sw128(r, byte);
            *reinterpret_cast<uint4*>(to) = make_uint4(q1[0], q1[1], q1[2], q1[3]);
            *reinterpret_cast<uint4*>(to + kChunks * kChunkBytes) = make_uint4(q2[0], q2[1], q2[2], q2[3]);
        };
#pragma unroll
        for (int m = 0; m < 8; ++m) store(l, 16 * m, y[m][0], y[m][1], y[m][2], y[m][3]);
        store(kRope, 16 * l, rope[0][0], rope[0][1], rope[1][0], rope[1][1]);
    }
}

// 32 bytes: one store where the address is a multiple of 32 (`wide`), which fills
// a sector at once, else two.
__device__ __forceinline__ void store32(void* dst, const uint32_t (&v)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        static_cast<uint4*>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        static_cast<uint4*>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

// A query vector's softmax state.
struct RowState {
    float m, R, E, logE, l;   // logE = inf: rows seen, but none with a latent scale yet
    float kept, lost;         // sum of this thread's weights, a quarter of the vector's before the
                              // last exact step; what their rounding may have lost
};

// What a softmax thread has summed up before the current kFold steps, in the workspace: its
// 128 columns of O, in the walker's second slot, its row sum l, and the factor that
// takes O's total to the current references.  Out of line and out of the step's registers:
// touched every kFold steps, and where an exact step follows the first of them.
struct Totals {
    float* o;
    float2* l;   // row sum, factor
};
__device__ __forceinline__ Totals totals_of(const PagedParams& p, int64_t pair, int rank, int tid) {
    const int vec = kHalf * rank + (tid & (kHalf - 1)), d0 = 256 * (tid >> 7) + 128 * ((tid >> 6) & 1);
    return {p.ws_o + ((2 * pair + 1) * kVecs + vec) * kMlaDV + d0, p.ws_l + (2 * pair + rank) * kSoft + tid};
}
// The accumulators (O from column `col`, l) into the totals, the first time or in addition.
static __device__ __noinline__ void fold_sums(const PagedParams& p, int64_t pair, int rank, uint32_t col, float l, bool first) {
    const Totals to = totals_of(p, pair, rank, threadIdx.x);
    const float2 had = first ? make_float2(0.0f, 0.0f) : *to.l;
    *to.l = make_float2(had.x + l, 1.0f);
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
        uint32_t o[16];
        tmem_ld16(col + 16 * c, o);
        tmem_wait_ld();
        float4* g = reinterpret_cast<float4*>(to.o + 16 * c);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 v = first ? make_float4(0.f, 0.f, 0.f, 0.f) : g[j];
            g[j] = make_float4(fmaf(v.x, had.y, __uint_as_float(o[4 * j])), fmaf(v.y, had.y, __uint_as_float(o[4 * j + 1])),
                               fmaf(v.z, had.y, __uint_as_float(o[4 * j + 2])), fmaf(v.w, had.y, __uint_as_float(o[4 * j + 3])));
        }
    }
}
// The totals back into O; returns l's.
static __device__ __noinline__ float unfold_sums(const PagedParams& p, int64_t pair, int rank, uint32_t col) {
    const Totals from = totals_of(p, pair, rank, threadIdx.x);
    const float2 had = *from.l;
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
        uint32_t o[16];
        tmem_ld16(col + 16 * c, o);
        tmem_wait_ld();
        const float4* g = reinterpret_cast<const float4*>(from.o + 16 * c);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 v = g[j];
            o[4 * j] = __float_as_uint(fmaf(v.x, had.y, __uint_as_float(o[4 * j])));
            o[4 * j + 1] = __float_as_uint(fmaf(v.y, had.y, __uint_as_float(o[4 * j + 1])));
            o[4 * j + 2] = __float_as_uint(fmaf(v.z, had.y, __uint_as_float(o[4 * j + 2])));
            o[4 * j + 3] = __float_as_uint(fmaf(v.w, had.y, __uint_as_float(o[4 * j + 3])));
        }
        tmem_st16(col + 16 * c, o);
    }
    tmem_wait_st();
    return had.x;
}
// The walk's current segment as a record; false at its end.
__device__ __forceinline__ bool announce(const PagedParams& p, const PagedWalk<PagedTensor>& walk, int64_t pair, Work* to) {
    Segment g;
    Work w{};
    const bool more = walk.get(p, g);
    if (more) {
        int64_t parts;
        w.steps = (int32_t)(g.u1 - g.u0);
        w.b = g.b;
        w.rows = g.rows;
        w.first = (int32_t)(g.u0 * kRows);
        w.end = (int32_t)row_limit(p, g, g.rows - 1);
        w.seen0 = (int32_t)row_limit(p, g, 0);
        w.row0 = g.row0;
        w.tok0 = g.tok0;
        w.base = g.base;
        w.slot = walk.slot(g, pair, &parts);
        w.parts = (int32_t)parts;
    }
    *to = w;
    return more;
}

template <bool TQ4>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    paged_tensor_kernel(const __grid_constant__ PagedParams p, const __grid_constant__ CUtensorMap map) {
    using R = Regs<TQ4>;
    launch_dependents();
    extern __shared__ __align__(1024) unsigned char sm[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kOffBar);
    volatile int* sAbort = reinterpret_cast<volatile int*>(sm + kOffMisc);
    uint32_t* sTmem = reinterpret_cast<uint32_t*>(sm + kOffMisc + 4);
    Work* sWork = reinterpret_cast<Work*>(sm + kOffWork);

    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFull, tid >> 5, 0);
    const int rank = (int)cta_rank();
    const int64_t pair = blockIdx.x >> 1;
    const int64_t wl = p.wait_limit;
    const bool aligned = (smem_u32(sm) & 1023u) == 0;   // else the swizzled operands would be misread

    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(sTmem)),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    if (tid == 64) {
        for (int i = 0; i < kNumBars; ++i) {
            const uint32_t count = i < kBarP          ? 2u * kDecWarps
                                   : i == kBarP       ? 2u * kSoftWarps
                                   : (i == kBarQ0 || i == kBarQ0 + 1) ? (uint32_t)kDecWarps
                                   : i == kBarOut     ? (uint32_t)kSoftWarps
                                   : (i == kBarWorkFree0 || i == kBarWorkFree0 + 1)
                                       ? (uint32_t)(kSoftWarps + kDecWarps + 1 + (TQ4 ? (rank == 0 ? 1 : 0) : 2))
                                   : (i == kBarScore0 || i == kBarScore0 + 1) ? 2u
                                   : (i == kBarScaleFree0 || i == kBarScaleFree0 + 1) ? (uint32_t)kSoftWarps
                                                                                      : 1u;
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(&bars[i])), "r"(count));
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *sAbort = aligned ? 0 : 1;
    }
    if (TQ4 && tid == 0) {
        uint32_t lo[2] = {0u, 0u}, hi[2] = {0u, 0u};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t h = __half_as_ushort(__float2half_rn(__fmul_rn(p.lv[8 + k], kGamma)));
            lo[k >> 2] |= (h & 0xffu) << (8 * (k & 3));
            hi[k >> 2] |= (h >> 8) << (8 * (k & 3));
        }
        *reinterpret_cast<uint4*>(sm + kOffLevels) = make_uint4(lo[0], lo[1], hi[0], hi[1]);
    }
    __syncwarp();
    cluster_arrive();
    grid_dependency_wait();
    if (rank == 0 && tid < 4) p.ws_desc[pair * 4 + tid] = 0;
    PagedWalk<PagedTensor> walk;
    // the same answer in both CTAs
    const bool any = walk.template start<kThreads>(p, pair, gridDim.x >> 1, reinterpret_cast<int64_t*>(sm + kOffPart));
    bool more = true;
    if (any && warp == kWalkWarp && lane == 0) more = announce(p, walk, pair, &sWork[0]);
    tc_before();
    __syncthreads();
    cluster_wait();   // the other CTA's barriers are there, its tensor memory is allocated
    tc_after();
    const uint32_t tmem = *sTmem;
    if (!any) {
        if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
        return;
    }

    if (warp >= kIssueWarp) {
        set_registers<R::kRest, R::kLaunch>();
        if (warp == kWalkWarp) {
            // ================= the walk: announces segments one ahead =================
            if (lane == 0) mbar_arrive(&bars[kBarWork0]);   // the first lies there
            more = __shfl_sync(kFull, (int)more, 0) != 0;
            for (int n = 1; more; ++n) {
                walk.next(p);
                if (lane == 0) {
                    // a wait of a segment's length, up to millions of steps
                    more = n < 2 || idle_wait(&bars[kBarWorkFree0 + (n & 1)], (uint32_t)(n / 2 - 1) & 1u, sAbort, 8 * wl);
                    if (more) {
                        more = announce(p, walk, pair, &sWork[n & 1]);
                        mbar_arrive(&bars[kBarWork0 + (n & 1)]);
                    }
                }
                more = __shfl_sync(kFull, (int)more, 0) != 0;
            }
        } else if (warp == kIssueWarp) {
            // ================= products (first CTA) =================
            if (rank == 0) {
                const uint64_t dq = umma_desc(smem_u32(sm + kOffQ), 16, 1024);
                const uint64_t dk = umma_desc(smem_u32(sm + kOffK), 16, 1024);
                const uint64_t dv = umma_desc(smem_u32(sm + kOffV), kVChunkBytes, 1024);
                const uint64_t dp = umma_desc(smem_u32(sm + kOffP), 16, 1024);
                constexpr uint64_t kStep = kChunkBytes >> 4, kVStep = kVChunkBytes >> 4, kSlotStep = kSlotBytes >> 4;
                const uint64_t dsk = umma_desc(smem_u32(sm + kOffSlot), 16, 1024);            // score rows
                const uint64_t dsv = umma_desc(smem_u32(sm + kOffSlot), kChunkBytes, 1024);   // context rows
                uint32_t fill = 0;   // TQ4: fills used so far
                bool ok = true;
                if (p.stall_polls > 0) ok = warp_wait(&bars[kBarNever], 0u, sAbort, p.stall_polls);
                auto scores = [&](uint32_t it) {
                    const uint32_t d = tmem + kColS + 128 * (it & 1u);
                    if (TQ4) {
#pragma unroll
                        for (int c = 0; c < kChunks; ++c) {
                            if (c % 3 == 0) {
                                if (!warp_wait(&bars[kBarFull0 + (fill & 1u)], (fill >> 1) & 1u, sAbort, wl)) return false;
                                tc_after();
                            }
                            const uint64_t ds = dsk + (fill & 1u) * kSlotStep + c % 3 * kStep;
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                                for (int part = 0; part < 2; ++part)
                                    pair_mma(d + (c < kRope ? 0 : 64), dq + (kChunks * part + c) * kStep + 2 * ks, ds + 2 * ks,
                                             kIdescScore, ((c > 0 && c < kRope) || ks > 0 || part > 0) ? 1u : 0u);
                            if (c % 3 == 2) pair_commit(&bars[kBarFree0 + (fill++ & 1u)]);
                        }
                    } else {
                        if (!warp_wait(&bars[kBarLat0 + (it & 1u)], (it >> 1) & 1u, sAbort, wl)) return false;
                        if (!warp_wait(&bars[kBarPeerLat0 + (it & 1u)], (it >> 1) & 1u, sAbort, wl)) return false;
                        tc_after();
                        const uint64_t dl = dk + (it & 1u) * 4 * kStep;
#pragma unroll
                        for (int kc = 0; kc < 4; ++kc)
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                                for (int part = 0; part < 2; ++part)
                                    pair_mma_f8(d, dq + (4 * part + kc) * kStep + 2 * ks, dl + kc * kStep + 2 * ks, kIdescScore,
                                                (kc > 0 || ks > 0 || part > 0) ? 1u : 0u);
                        if (!warp_wait(&bars[kBarRope], it & 1u, sAbort, wl)) return false;
                        if (!warp_wait(&bars[kBarPeerRope], it & 1u, sAbort, wl)) return false;
                        tc_after();
#pragma unroll
                        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                            for (int part = 0; part < 2; ++part)
                                pair_mma_f8(d + 64, dq + kRope * kStep + 4 * part + 2 * ks, dk + kRope * kStep + 4 + 2 * ks,
                                            kIdescScore, (ks > 0 || part > 0) ? 1u : 0u);
                    }
                    pair_commit(&bars[kBarScore0 + (it & 1u)]);
                    return true;
                };
                uint32_t it = 0;   // step of the whole walk
                for (int n = 0; ok; ++n) {
                    ok = warp_wait(&bars[kBarWork0 + (n & 1)], (uint32_t)(n >> 1) & 1u, sAbort, wl);
                    if (!ok) break;
                    const int steps = __shfl_sync(kFull, sWork[n & 1].steps, 0);
                    warp_arrive(&bars[kBarWorkFree0 + (n & 1)], lane);
                    if (steps == 0) break;
                    if (!TQ4) {   // TQ4: the score rows come after the queries of the same warps
                        ok = warp_wait(&bars[kBarQFirst], (uint32_t)n & 1u, sAbort, wl);
                        if (!ok) break;
                    }
                    // scores of step t, then the context of step t - 1; the other score
                    // buffer is free by then, as its weights came before the last context
                    for (int t = 0; t <= steps && ok; ++t) {
                        if (t < steps && !(ok = scores(it + t))) break;
                        if (t == 0) continue;
                        const uint32_t s = it + t - 1;   // step of the context
                        ok = warp_wait(&bars[kBarP], s & 1u, sAbort, wl);
                        if (!ok) break;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            ok = ok && (TQ4 ? warp_wait(&bars[kBarFull0 + (fill & 1u)], (fill >> 1) & 1u, sAbort, wl)
                                            : warp_wait(&bars[kBarV0 + h], s & 1u, sAbort, wl));
                            if (!ok) break;
                            tc_after();
                            const uint64_t dh = TQ4 ? dsv + (fill & 1u) * kSlotStep : dv + 4 * h * 128;
#pragma unroll
                            for (int j = 0; j < 2; ++j)
#pragma unroll
                                for (int ks = 0; ks < 4; ++ks)
                                    pair_mma(tmem + kColO + 128 * j, dp + h * kStep + 2 * ks,
                                             dh + 2 * j * (TQ4 ? kStep : kVStep) + ks * 128, kIdescCtx,
                                             ((t - 1) % kFold > 0 || h > 0 || ks > 0) ? 1u : 0u);
                            if (TQ4) pair_commit(&bars[kBarFree0 + (fill++ & 1u)]);
                            if (!TQ4 || h == 1) pair_commit(&bars[kBarCtx0 + h]);
                        }
                    }
                    it += steps;
                }
                __syncwarp();
                pair_commit(&bars[kBarDone]);
            } else if (!TQ4) {
                // ================= this CTA's codes are there: tell the first =================
                uint32_t it = 0;
                bool ok = true;
                for (int n = 0; ok; ++n) {
                    if (!(ok = warp_wait(&bars[kBarWork0 + (n & 1)], (uint32_t)(n >> 1) & 1u, sAbort, wl))) break;
                    const int steps = __shfl_sync(kFull, sWork[n & 1].steps, 0);
                    warp_arrive(&bars[kBarWorkFree0 + (n & 1)], lane);
                    if (steps == 0) break;
                    for (int t = 0; t < steps && ok; ++t, ++it) {
                        if (!(ok = warp_wait(&bars[kBarLat0 + (it & 1u)], (it >> 1) & 1u, sAbort, wl))) break;
                        warp_arrive_first(&bars[kBarPeerLat0 + (it & 1u)], lane);
                        if (!(ok = warp_wait(&bars[kBarRope], it & 1u, sAbort, wl))) break;
                        warp_arrive_first(&bars[kBarPeerRope], lane);
                    }
                }
            }
        } else if (warp == kLoadWarp) {
            if (!TQ4) {
                // ================= codes of the score rows, by TMA =================
                // this CTA's 64 rows of a step in boxes of whole pages (64 rows at
                // most): lanes 0-15 a box and 128 latent dims each, lanes 16-19 a box's
                // last 128 bytes.  Boxes past the sequence's end are left as they are:
                // the softmax drops their scores.
                const int box = min(1 << p.shift, kHalf);
                const int j = lane < 16 ? lane >> 2 : lane - 16, c = lane < 16 ? lane & 3 : 0;
                const bool mine = lane < 20 && j * box < kHalf;
                uint32_t it = 0, lat = 0, rope = 0;   // steps; steps whose latent, whose rope codes were asked for
                bool ok = true;
                for (int n = 0; ok; ++n) {
                    if (!(ok = warp_wait(&bars[kBarWork0 + (n & 1)], (uint32_t)(n >> 1) & 1u, sAbort, wl))) break;
                    const Work w = sWork[n & 1];
                    warp_arrive(&bars[kBarWorkFree0 + (n & 1)], lane);
                    if (w.steps == 0) break;
                    const int32_t* table = p.table + (int64_t)w.b * p.table_stride;
                    const int32_t row0 = w.first + kHalf * rank + j * box;
                    auto page = [&](int t) {
                        const int32_t r = row0 + t * kRows;
                        return mine && t < w.steps && r < w.end ? table[r >> p.shift] : 0;
                    };
                    int32_t id = page(0);
                    for (int t = 0; t < w.steps; ++t, ++it) {
                        const int32_t r = row0 + t * kRows;
                        const bool live = mine && r < w.end;
                        if (id < 0 || id >= p.n_pages) id = 0;   // the decode warps report it
                        const int32_t y = (id << p.shift) + (r & ((1 << p.shift) - 1));
                        const uint32_t boxes = __popc(__ballot_sync(kFull, live && lane >= 16));
                        id = page(t + 1);
                        if (it >= 2 && !(ok = warp_wait(&bars[kBarScore0 + (it & 1u)], (it / 2 - 1) & 1u, sAbort, wl))) break;
                        if (lane == 0) expect_bytes(&bars[kBarLat0 + (it & 1u)], boxes * box * 512);
                        ++lat;
                        __syncwarp();
                        if (live && lane < 16)
                            load_box(sm + kOffK + (4 * (it & 1u) + c) * kChunkBytes + j * box * 128, &map, 128 * c, y,
                                     &bars[kBarLat0 + (it & 1u)]);
                        if (it >= 1 && !(ok = warp_wait(&bars[kBarScore0 + ((it - 1) & 1u)], ((it - 1) >> 1) & 1u, sAbort, wl)))
                            break;
                        if (lane == 0) expect_bytes(&bars[kBarRope], boxes * box * 128);
                        ++rope;
                        __syncwarp();
                        if (live && lane >= 16)
                            load_box(sm + kOffK + kRope * kChunkBytes + j * box * 128, &map, kMlaD - 128, y, &bars[kBarRope]);
                    }
                }
                // after an abort too, no copy outlives the CTA's shared memory
                volatile int never = 0;
                for (uint32_t k = lat > 2 ? lat - 2 : 0; k < lat; ++k)
                    mbar_wait(&bars[kBarLat0 + (k & 1u)], (k >> 1) & 1u, &never, kWaitLimit);
                if (rope > 0) mbar_wait(&bars[kBarRope], (rope - 1) & 1u, &never, kWaitLimit);
            }
        } else if (warp == kScaleWarp) {
            // ================= row scales, two steps ahead =================
            // 4 consecutive rows a lane: in one page, as pages hold whole multiples of 16
            uint32_t it = 0;
            bool ok = true;
            for (int n = 0; ok; ++n) {
                if (!(ok = warp_wait(&bars[kBarWork0 + (n & 1)], (uint32_t)(n >> 1) & 1u, sAbort, wl))) break;
                const Work w = sWork[n & 1];
                warp_arrive(&bars[kBarWorkFree0 + (n & 1)], lane);
                if (w.steps == 0) break;
                const int32_t* table = p.table + (int64_t)w.b * p.table_stride;
                auto page = [&](int t) {
                    const int32_t x = w.first + t * kRows + 4 * lane;
                    return t < w.steps && x < w.end ? table[x >> p.shift] : 0;
                };
                int32_t id = page(0);
                for (int t = 0; t < w.steps; ++t, ++it) {
                    const int32_t x = w.first + t * kRows + 4 * lane;
                    if (id < 0 || id >= p.n_pages) id = 0;   // the decode warps report it
                    const float* s = p.scales + (((int64_t)id << p.shift) + (x & ((1 << p.shift) - 1))) * p.n_blocks;
                    float2 v[4];
                    float top = 0.0f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[i] = make_float2(0.f, 0.f);
                        if (x + i < w.end) v[i] = make_float2(s[i * p.n_blocks], s[(i + 1) * p.n_blocks - 1]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = row_scales(v[i].x, v[i].y);
                    id = page(t + 1);
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = fmaxf(top, v[i].x);
                    top = warp_max(top);
                    if (it >= 2 && !(ok = warp_wait(&bars[kBarScaleFree0 + (it & 1u)], (it / 2 - 1) & 1u, sAbort, wl))) break;
                    float4* dst = reinterpret_cast<float4*>(sm + kOffScale + (it & 1u) * kScaleBytes) + lane;
                    dst[0] = make_float4(v[0].x, v[1].x, v[2].x, v[3].x);
                    dst[kRows / 4] = make_float4(v[0].y, v[1].y, v[2].y, v[3].y);
                    if (lane == 0) reinterpret_cast<float*>(sm + kOffMax)[it & 1u] = top > 0.0f ? __log2f(top) : -INFINITY;
                    warp_arrive(&bars[kBarScore0 + (it & 1u)], lane);
                }
            }
        }
    } else if (warp >= kSoftWarps) {
        // ================= decode warps =================
        set_registers<R::kDecode, R::kLaunch>();
        const int dw = warp - kSoftWarps;
        uint32_t it = 0;
        bool ok = true;
        for (int n = 0; ok; ++n) {
            if (!(ok = warp_wait(&bars[kBarWork0 + (n & 1)], (uint32_t)(n >> 1) & 1u, sAbort, wl))) break;
            const Work& work = sWork[n & 1];
            const int32_t steps = work.steps, first = work.first, end = work.end, rows = work.rows;
            const int64_t row0 = work.row0;
            const int32_t* table = p.table + (int64_t)work.b * p.table_stride;
            warp_arrive(&bars[kBarWorkFree0 + (n & 1)], lane);
            if (steps == 0) break;
            // pages are asked for a step before the codes, the codes a step before their use
            auto page = [&](int32_t r) { return r < end ? table[r >> p.shift] : 0; };
            auto code_rows = [&](int32_t r, int32_t id) {
                if (id < 0 || id >= p.n_pages) {
                    if (lane == 0 && r < end) set_err(p.err, KVQ_ERR_ARG);
                    id = 0;
                }
                return p.codes + (((int64_t)id << p.shift) + (r & ((1 << p.shift) - 1))) * (TQ4 ? kMlaD / 2 : kMlaD);
            };
            // the scores of the last segment have read its queries
            if (it > 0 && !(ok = warp_wait(&bars[kBarScore0 + ((it - 1) & 1u)], ((it - 1) >> 1) & 1u, sAbort, wl))) break;
            float* cz = reinterpret_cast<float*>(sm + kOffCz) + (n & 1) * kHalf;
            if (TQ4)
                rotate_queries(p, row0 + kHalf * rank, rows - kHalf * rank, sm + kOffQ, cz, dw, lane);
            else
                load_queries(p, row0 + kHalf * rank, rows - kHalf * rank, sm + kOffQ, cz, dw, lane);
            fence_async_smem();
            warp_arrive(&bars[kBarQ0 + (n & 1)], lane);
            if (!TQ4) warp_arrive_first(&bars[kBarQFirst], lane);
            // the context rows' place staged the last segment's output
            auto stage_free = [&]() { return n == 0 || warp_wait(&bars[kBarOut], (uint32_t)(n - 1) & 1u, sAbort, wl); };
            if constexpr (TQ4) {
                const uint4 lv = *reinterpret_cast<const uint4*>(sm + kOffLevels);
                const Planes pl{{lv.x, lv.y}, {lv.z, lv.w}};
                constexpr int kRowBytes = kMlaD / 2;
                // A warp has 8 consecutive rows (they lie in one page) of the own 64 for the
                // scores, and of both halves of the step for the context:
                //   score rows: row lane / 4, of each chunk the quarter lane % 4 (8 bytes)
                //   context rows: rows 4 i + lane / 2 % 4, chunk lane / 8, half lane % 2 (16 bytes)
                // so that the 8 lanes of a store have different 16-byte units.  The codes of
                // the own half come twice (L2 has room, 10% busy).  The next step's are asked for
                // fill by fill, into the registers that have just been stored (256 tokens on
                // 16,384 rows 1.73 ms, 1.80 with all of a kind at once).
                const int k_row = lane >> 2, k_quarter = lane & 3;
                const int v_row = (lane >> 1) & 3, v_half = lane & 1, v_chunk = lane >> 3;
                const int k_byte = k_row * kRowBytes + 8 * k_quarter;
                const int v_byte = v_row * kRowBytes + 128 * (v_chunk >> 1) + 64 * rank + 32 * (v_chunk & 1) + 16 * v_half;
                const int32_t row_k = first + kHalf * rank + 8 * dw, row_v = first + 8 * dw;
                uint32_t fill = 5 * it;   // fills so far
                int32_t id_k = page(row_k), id_v[2] = {page(row_v), page(row_v + kHalf)};
                uint2 k[kChunks];
                uint4 v[2][2];
                const uint8_t* from_k = nullptr;   // this lane's codes of the step that is asked for
                bool there_k = false;
                auto step_k = [&](int t) {
                    const int32_t r = row_k + t * kRows;
                    from_k = code_rows(r, id_k) + k_byte;
                    there_k = t < steps && r + k_row < end;
                    id_k = t + 1 < steps ? page(r + kRows) : 0;
                };
                auto request_k = [&](int g) {   // chunks 3 g ..
#pragma unroll
                    for (int c = 3 * g; c < 3 * g + 3; ++c)
                        k[c] = there_k ? *reinterpret_cast<const uint2*>(from_k + 32 * c) : make_uint2(0u, 0u);
                };
                auto request_v = [&](int t, int h) {   // rows 64 h ..
                    const int32_t r = row_v + t * kRows + kHalf * h;
                    const uint8_t* a = code_rows(r, id_v[h]) + v_byte;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        v[h][i] = t < steps && r + 4 * i + v_row < end
                                      ? *reinterpret_cast<const uint4*>(a + 4 * i * kRowBytes)
                                      : make_uint4(0u, 0u, 0u, 0u);
                    id_v[h] = t + 1 < steps ? page(r + kRows) : 0;
                };
                // A wait that runs out ends the loop with the step; from there on nothing is stored
                // (the slot may still be read) or handed over.
                auto begin = [&]() {
                    if (fill >= 2 && !warp_wait(&bars[kBarFree0 + (fill & 1u)], ((fill >> 1) - 1) & 1u, sAbort, wl)) ok = false;
                    return sm + kOffSlot + (fill & 1u) * kSlotBytes;
                };
                auto finish = [&]() {
                    fence_async_smem();
                    if (ok) warp_arrive_first(&bars[kBarFull0 + (fill & 1u)], lane);
                    ++fill;
                };
                step_k(0);
#pragma unroll
                for (int g = 0; g < 3; ++g) request_k(g);
                request_v(0, 0);
                request_v(0, 1);
                if (!(ok = stage_free())) break;
                // score rows of step t, then context rows of step t - 1
                for (int t = 0; t <= steps; ++t) {
                    if (t < steps) {
                        step_k(t + 1);
#pragma unroll
                        for (int g = 0; g < 3; ++g) {
                            unsigned char* to = begin();
                            if (ok) {
#pragma unroll
                                for (int c = 0; c < 3; ++c) {
                                    store_levels(to + c * kChunkBytes, k[3 * g + c].x, 8 * dw + k_row, 2 * k_quarter, pl);
                                    store_levels(to + c * kChunkBytes, k[3 * g + c].y, 8 * dw + k_row, 2 * k_quarter + 1, pl);
                                }
                            }
                            finish();
                            request_k(g);
                        }
                    }
                    if (t == 0) continue;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        unsigned char* to = begin() + v_chunk * kChunkBytes;
                        if (ok) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t in[4] = {v[h][i].x, v[h][i].y, v[h][i].z, v[h][i].w};
#pragma unroll
                                for (int u = 0; u < 4; ++u) store_levels(to, in[u], 8 * dw + 4 * i + v_row, 4 * v_half + u, pl);
                            }
                        }
                        finish();
                        request_v(t, h);
                    }
                    if (!ok) break;
                }
            } else {
                // Context rows: a warp has 8 consecutive rows of each half of a step (8 rows
                // lie in one page): rows 2 i, 2 i + 1, bit 2 of the lane picks the row, lane / 8
                // the chunk, lane % 4 the quarter.
                const int q4 = lane & 3, up = (lane >> 2) & 1, c4 = lane >> 3;
                unsigned char* v_chunk = sm + kOffV + c4 * kVChunkBytes;
                const int v_piece = 16 * (c4 >> 1) + 8 * rank + 4 * (c4 & 1) + q4;   // of the row's 36
                const int32_t row_v = first + 8 * dw;
                int32_t id_v[2] = {page(row_v), page(row_v + kHalf)};
                uint4 ctx[2][4];
                auto request_v = [&](int t) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int32_t r0 = row_v + t * kRows + kHalf * h;
                        const uint8_t* a = code_rows(r0, id_v[h]) + up * kMlaD + 16 * v_piece;
                        const int last = end - r0 - up;   // rows 2 i up to here exist
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            ctx[h][i] = 2 * i < last ? ldg16(a + 2 * i * kMlaD) : make_uint4(0u, 0u, 0u, 0u);
                        if (t + 1 < steps) id_v[h] = page(r0 + kRows);
                    }
                };
                request_v(0);
                if (!(ok = stage_free())) break;
                for (int t = 0; t < steps && ok; ++t) {
                    const uint32_t s = it + t;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (s > 0 && !(ok = warp_wait(&bars[kBarCtx0 + h], (s - 1) & 1u, sAbort, wl))) break;
#pragma unroll
                        for (int i = 0; i < 4; ++i) store_codes(v_chunk, ctx[h][i], kHalf * h + 8 * dw + 2 * i + up, q4);
                        fence_async_smem();
                        warp_arrive_first(&bars[kBarV0 + h], lane);
                    }
                    if (ok && t + 1 < steps) request_v(t + 1);
                }
            }
            it += steps;
        }
    } else {
        // ================= softmax warps =================
        set_registers<R::kSoftmax, R::kLaunch>();
        // vector (of this CTA); rows 64 half + 32 sub .. + 31 of a step
        const int r = tid & (kHalf - 1), half = (tid >> 6) & 1, sub = tid >> 7;
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        unsigned char* sP = sm + kOffP + half * kChunkBytes;
        // between the four threads of a vector: the weights' buffer, while no step's
        // weights are in it; a group's part of it, while none of its own are
        float* sX = reinterpret_cast<float*>(sm + kOffP);
        const int group = warp & 1;
        float* gX = reinterpret_cast<float*>(sm + kOffP + 32 * 128 * group);
        uint32_t it = 0;
        bool aborted = false;
        for (int n = 0;; ++n) {
            if (!warp_wait(&bars[kBarWork0 + (n & 1)], (uint32_t)(n >> 1) & 1u, sAbort, wl)) aborted = true;
            if (worker_any<kSoft>(aborted)) {
                aborted = true;
                break;
            }
            const Work& w = sWork[n & 1];
            const int steps = w.steps;
            if (steps == 0) break;
            const int32_t first = w.first, seen0 = w.seen0;
            // vectors past the tile's last repeat its limit: they score 0 and are dropped
            const int vec = kHalf * rank + r;
            const int32_t lim = (int32_t)max((int64_t)0, w.base + 1 + over_heads(p, w.tok0 + min(vec, w.rows - 1)));
            RowState st{-INFINITY, -INFINITY, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            if (!warp_wait(&bars[kBarQ0 + (n & 1)], (uint32_t)(n >> 1) & 1u, sAbort, wl)) aborted = true;
            const float cz = reinterpret_cast<const float*>(sm + kOffCz)[(n & 1) * kHalf + r];
            int t = 0;
            for (int until = min(steps, kFold);; until = min(steps, until + kFold)) {
                for (; t < until; ++t, ++it) {
                    warp_wait(&bars[kBarScore0 + (it & 1u)], (it >> 1) & 1u, sAbort, wl);
                    tc_after();
                    const float* s_l = reinterpret_cast<const float*>(sm + kOffScale + (it & 1u) * kScaleBytes) + kHalf * half +
                                       kCols * sub;
                    const int seen_abort = *sAbort;   // read ahead of its use
                    const float log_s = reinterpret_cast<const float*>(sm + kOffMax)[it & 1u];   // of the step's largest s_L
                    const uint32_t ts = tmem + lane_base + kColS + 128 * (it & 1u) + kCols * sub;
                    const int32_t t0 = first + t * kRows + kHalf * half + kCols * sub;
                    const bool masked = first + (t + 1) * kRows > seen0;
                    float z[kCols];
                    float4 s_lat[kCols / 4];
                    auto scores = [&](float ref) {   // z - ref of this thread's rows
                        const F2 cz2 = f2(cz, cz), ref2 = f2(-ref, -ref);
#pragma unroll
                        for (int c = 0; c < kCols; c += 16) {
                            uint32_t a[16], b[16];
                            tmem_ld16(ts + c, a);
                            tmem_ld16(ts + 64 + c, b);
                            float4 s_r[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                s_lat[c / 4 + j] = *reinterpret_cast<const float4*>(s_l + c + 4 * j);
                                s_r[j] = *reinterpret_cast<const float4*>(s_l + kRows + c + 4 * j);
                            }
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; j += 4) {
                                const float4 sl = s_lat[(c + j) / 4], sr = s_r[j / 4];
                                const F2 z0 = fma2(fma2(f2(a[j], a[j + 1]), f2(sl.x, sl.y), mul2(f2(b[j], b[j + 1]), f2(sr.x, sr.y))),
                                                   cz2, ref2);
                                const F2 z1 = fma2(
                                    fma2(f2(a[j + 2], a[j + 3]), f2(sl.z, sl.w), mul2(f2(b[j + 2], b[j + 3]), f2(sr.z, sr.w))), cz2,
                                    ref2);
                                const float2 u0 = unpack(z0), u1 = unpack(z1);
                                z[c + j] = u0.x;
                                z[c + j + 1] = u0.y;
                                z[c + j + 2] = u1.x;
                                z[c + j + 3] = u1.y;
                            }
                        }
                        if (masked) {
#pragma unroll
                            for (int j = 0; j < kCols; ++j)
                                if (t0 + j >= lim) z[j] = -INFINITY;
                        }
                    };
                    // The first step has no reference yet and goes to the exact path with
                    // plain scores; a later one comes back for them if a vote sends it there.
                    const bool low = st.lost > kLossShare * st.kept;   // (NaN: no)
                    bool exact = t == 0, stop = false;
                    for (;;) {
                        scores(exact ? 0.0f : st.m);
                        if (!exact) {
                            float top[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
                            for (int j = 4; j < kCols; ++j) top[j & 3] = fmaxf(top[j & 3], z[j]);
                            const float dmax = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                            const float log_se = log_s + st.logE;
                            const bool flag = aborted | (seen_abort != 0) | (dmax + log_se > kLogWmax) | (dmax > kLogMax) |
                                              (log_se > kLogMax) | low;
                            if (!group_any(group, flag)) break;
                            exact = true;
                            continue;
                        }
                        // ---- exact path: row maxima, new references, O rescaled ----
                        if (it > 0 && !warp_wait(&bars[kBarCtx0 + 1], (it - 1) & 1u, sAbort, wl)) aborted = true;
                        if (group_any(group, aborted | (*sAbort != 0))) {
                            stop = true;
                            break;
                        }
                        tc_after();
                        float zt = -INFINITY, yt = -INFINITY;
#pragma unroll
                        for (int j = 0; j < kCols; j += 4) {
                            const float4 sl = TQ4 ? *reinterpret_cast<const float4*>(s_l + j) : s_lat[j / 4];
                            const float s[4] = {sl.x, sl.y, sl.z, sl.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                zt = fmaxf(zt, z[j + k]);
                                yt = fmaxf(yt, z[j + k] + (s[k] > 0.0f ? __log2f(s[k]) : -INFINITY));   // -inf: an inert latent block
                            }
                        }
                        gX[32 * (warp >> 1) + lane] = zt;
                        gX[128 + 32 * (warp >> 1) + lane] = yt;
                        gX[256 + 32 * (warp >> 1) + lane] = low ? -st.kept : st.kept;
                        group_sync(group);
                        float kept = 0.0f;
                        bool fall = false;   // the same in all four
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            zt = fmaxf(zt, gX[32 * k + lane]);
                            yt = fmaxf(yt, gX[128 + 32 * k + lane]);
                            const float w = gX[256 + 32 * k + lane];
                            kept += fabsf(w);
                            fall |= __float_as_int(w) < 0;
                        }
                        group_sync(group);   // read before any thread's weights go there
                        const float mn = fmaxf(st.m, zt), rn = fmaxf(fall ? st.R - kMaxDrop : st.R, yt);
                        const bool inert = rn == -INFINITY;
                        float le = fminf(mn - rn - kHeadroom, fminf(kLogEmax, kLogMax - log_s));   // s_L E stays finite
                        const float al = st.m == -INFINITY ? 0.0f : ex2(st.m - mn);
                        // O holds sum p s_L E c: rescaled by (E_new / E_old) 2^(m_old - m_new)
                        const float ao = st.R == -INFINITY ? 0.0f : ex2(le - st.logE + (st.m - mn));
                        // the weights are shared out, and this step's largest counts in all four threads
                        st.kept = inert ? 0.0f : 0.25f * fmaf(kept, ao, ex2(yt + (le - mn)));
                        st.lost *= ao;
                        if (fall) st.lost = fminf(st.lost, 0.9375f * kLossShare * st.kept);
                        st.l *= al;
                        if (t >= kFold) {
                            float2* had = totals_of(p, pair, rank, tid).l;
                            *had = make_float2(had->x * al, had->y * ao);
                        }
                        st.m = mn;
                        st.R = rn;
                        // rows seen without a latent scale: the next one comes here again;
                        // no row seen: the first score does, by m = -inf
                        st.logE = inert && mn > -INFINITY ? INFINITY : le;
                        st.E = inert ? 0.0f : ex2(le);
                        if (t > 0) {   // (to no use where this step's product starts from zero)
#pragma unroll 1
                            for (int c = 8 * sub; c < 8 * sub + 8; ++c) {   // 128 of the columns a thread
                                uint32_t o[16];
                                tmem_ld16(tmem + lane_base + kColO + 16 * c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * ao);
                                tmem_st16(tmem + lane_base + kColO + 16 * c, o);
                            }
                            tmem_wait_st();
                            if (warp < 2 && lane == 0) atomicAdd(p.exact_count, 1u);
                        }
                        // a vector that has seen no row keeps z = -inf
                        const float ref = mn == -INFINITY ? 0.0f : mn;
#pragma unroll
                        for (int j = 0; j < kCols; ++j) z[j] -= ref;
                        break;
                    }
                    if (stop) {
                        aborted = true;
                        break;
                    }
                    // asked before the weights are computed, used after: has the context
                    // of the step before read its weights?
                    const bool free_p = it == 0 || try_once(smem_u32(&bars[kBarCtx0 + 1]), (it - 1) & 1u);
                    uint32_t pk[kCols / 2];
                    F2 sum2 = f2(0.0f, 0.0f), kept2 = f2(0.0f, 0.0f);
                    const F2 e2 = f2(st.E, st.E);
#pragma unroll
                    for (int j = 0; j < kCols; j += 4) {
                        const float4 sl = TQ4 ? *reinterpret_cast<const float4*>(s_l + j) : s_lat[j / 4];
                        const float e[4] = {ex2(z[j]), ex2(z[j + 1]), ex2(z[j + 2]), ex2(z[j + 3])};
                        const F2 p0 = f2(e[0], e[1]), p1 = f2(e[2], e[3]);
                        sum2 = add2(sum2, add2(p0, p1));
                        const F2 x0 = mul2(p0, mul2(e2, f2(sl.x, sl.y))), x1 = mul2(p1, mul2(e2, f2(sl.z, sl.w)));
                        kept2 = add2(kept2, add2(x0, x1));
                        const float2 w0 = unpack(x0), w1 = unpack(x1);
                        const __half2 h0 = __floats2half2_rn(w0.x, w0.y), h1 = __floats2half2_rn(w1.x, w1.y);
                        pk[j / 2] = *reinterpret_cast<const uint32_t*>(&h0);
                        pk[j / 2 + 1] = *reinterpret_cast<const uint32_t*>(&h1);
                    }
                    const float2 sum = unpack(sum2);
                    st.l += sum.x + sum.y;
                    const float2 kept = unpack(kept2);
                    st.kept += kept.x + kept.y;
                    st.lost = st.E > 0.0f ? st.lost + kLossStep : 0.0f;
                    warp_arrive(&bars[kBarScaleFree0 + (it & 1u)], lane);
                    if (!__all_sync(kFull, free_p)) warp_wait(&bars[kBarCtx0 + 1], (it - 1) & 1u, sAbort, wl);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<uint4*>(sP + sw128(r, 64 * sub + 16 * i)) =
                            make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
                    fence_async_smem();
                    tc_before();
                    warp_arrive_first(&bars[kBarP], lane);
                }
                if (aborted || t == steps) break;
                // ---- the next product starts from zero ----
                // (a wait that runs out in one warp alone is told to the others by the next vote:
                // warps that part here would wait for one another at different barriers)
                if (warp_wait(&bars[kBarCtx0 + 1], (it - 1) & 1u, sAbort, wl)) {
                    tc_after();
                    fold_sums(p, pair, rank, tmem + lane_base + kColO + 128 * sub, st.l, t == kFold);
                    st.l = 0.0f;
                } else {
                    aborted = true;
                }
            }
            // ---- output ----
            if (!aborted && !warp_wait(&bars[kBarCtx0 + 1], (it - 1) & 1u, sAbort, wl)) aborted = true;
            if (worker_any<kSoft>(aborted)) {
                aborted = true;
                break;
            }
            tc_after();
            if (steps > kFold) st.l += unfold_sums(p, pair, rank, tmem + lane_base + kColO + 128 * sub);
            sX[tid] = st.l;
            worker_sync<kSoft>();
            const float l = (sX[r] + sX[kHalf + r]) + (sX[2 * kHalf + r] + sX[3 * kHalf + r]);   // the same in all four
            worker_sync<kSoft>();
            const int64_t slot = w.slot;
            float f = st.R == -INFINITY ? 0.0f : ex2(-st.logE);
            if (TQ4) f *= 1.0f / kGamma;
            if (slot < 0) f = l == 0.0f ? 0.0f : f / l;   // no visible row: zeros
            if (slot >= 0 && tid < kHalf) {
                float* ml = p.ws_ml + (slot * kVecs + vec) * 2;
                ml[0] = st.m * kLn2;
                ml[1] = l;
            }
            if (rank == 0 && tid == 0 && w.parts > 0) {
                p.ws_desc[pair * 4] = w.parts;
                p.ws_desc[pair * 4 + 1] = w.row0;
                p.ws_desc[pair * 4 + 2] = w.rows;
            }
            // dims d0 + 16 c .. + 15 of this vector, c < 8
            const int d0 = 256 * sub + 128 * half;
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + w.row0 * kMlaDV;
            const int rows = w.rows;
            const bool wide = (((uintptr_t)p.out | (uintptr_t)p.ws_o) & 31) == 0;
            auto context = [&](int c, float (&o)[16]) {
                uint32_t u[16];
                tmem_ld16(tmem + lane_base + kColO + 128 * sub + 16 * c, u);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __uint_as_float(u[j]) * f;
            };
            if (slot >= 0) {
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                    float o[16];
                    context(c, o);
                    float* dst = p.ws_o + (slot * kVecs + vec) * kMlaDV + d0 + 16 * c;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t u[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(o[8 * h + i]);
                        store32(dst + 8 * h, u, wide);
                    }
                }
            } else if (!TQ4) {
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                    float o[16];
                    context(c, o);
                    uint32_t h[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const __nv_bfloat162 b2 = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
                        h[i] = *reinterpret_cast<const uint32_t*>(&b2);
                    }
                    if (vec < rows) store32(out + (int64_t)vec * kMlaDV + d0 + 16 * c, h, wide);
                }
            } else {
                // unrotate: 32 vectors at a time through the context buffer (free
                // until the next segment's rows), 16-byte units swizzled by vector.
                // The 5 stages within 32 dims in the vector's own threads, the 4 over
                // them by 8 lanes a vector.
                float* stage = reinterpret_cast<float*>(sm + kOffV);
#pragma unroll 1
                for (int rr = 0; rr < 2; ++rr) {
                    if ((r >> 5) == rr) {
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t u[32];
                            F2 x[8][2];
                            tmem_ld32(tmem + lane_base + kColO + 128 * sub + 32 * c, u);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                x[i][0] = mul2(f2(u[4 * i], u[4 * i + 1]), f2(f, f));
                                x[i][1] = mul2(f2(u[4 * i + 2], u[4 * i + 3]), f2(f, f));
                            }
                            transform_in(x);
                            transform_over(x);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float2 a = unpack(x[i][0]), b = unpack(x[i][1]);
                                *reinterpret_cast<float4*>(stage + lane * kMlaDV + 4 * ((d0 / 4 + 8 * c + i) ^ (lane & 7))) =
                                    make_float4(a.x, a.y, b.x, b.y);
                            }
                        }
                    }
                    worker_sync<kSoft>();
                    {
                        const int k = 4 * warp + (lane >> 3), l = lane & 7;
                        const int ov = kHalf * rank + 32 * rr + k;
                        F2 x[16][2];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float4 y = *reinterpret_cast<const float4*>(stage + k * kMlaDV + 4 * ((l + 8 * i) ^ (k & 7)));
                            x[i][0] = f2(y.x, y.y);
                            x[i][1] = f2(y.z, y.w);
                        }
                        transform_over(x);
                        float v[16][4];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 a = unpack(x[i][0]), b = unpack(x[i][1]);
                            v[i][0] = a.x;
                            v[i][1] = a.y;
                            v[i][2] = b.x;
                            v[i][3] = b.y;
                        }
                        apply_signs(v, p.signs.w, l);
                        if (ov < rows) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const __nv_bfloat162 a = __floats2bfloat162_rn(v[i][0] * p.kn[0], v[i][1] * p.kn[0]);
                                const __nv_bfloat162 b = __floats2bfloat162_rn(v[i][2] * p.kn[0], v[i][3] * p.kn[0]);
                                *reinterpret_cast<uint2*>(out + (int64_t)ov * kMlaDV + 4 * (l + 8 * i)) =
                                    make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
                            }
                        }
                    }
                    worker_sync<kSoft>();
                }
            }
            tc_before();
            warp_arrive(&bars[kBarOut], lane);
            warp_arrive(&bars[kBarWorkFree0 + (n & 1)], lane);
        }
        // bounded, and not cut short by the abort flag: tensor memory is
        // released only after the products in flight have completed
        volatile int never = 0;
        if (!mbar_wait(&bars[kBarDone], 0u, &never, kWaitLimit)) aborted = true;
        if ((aborted || *sAbort != 0) && tid == 0) set_err(p.err, aligned ? KVQ_ERR_TIMEOUT : KVQ_ERR_DEVICE);
    }
    __syncwarp();
    tc_before();
    __syncthreads();
    cluster_sync();   // nothing of either CTA is in flight towards the other
    tc_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
}

// The pool as a matrix of bytes, read in boxes of 128 bytes x `box` rows in the
// 128-byte swizzle.
cudaError_t pool_map(const PagedParams& p, CUtensorMap* map) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e =
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)kMlaD, (cuuint64_t)p.n_pages << p.shift};
    const cuuint64_t strides[1] = {(cuuint64_t)kMlaD};
    const cuuint32_t box[2] = {128, (cuuint32_t)(1 << p.shift < kHalf ? 1 << p.shift : kHalf)}, step[2] = {1, 1};
    const CUresult r = reinterpret_cast<Encode>(fn)(
        map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p.codes), dims, strides, box, step,
        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <bool TQ4>
cudaError_t launch(const PagedParams& p, cudaStream_t stream) {
    // a setmaxnreg.inc waits for registers that other warps have released:
    // launch only if the split adds up against the launch's own count
    cudaFuncAttributes fa{};
    cudaError_t e = cudaFuncGetAttributes(&fa, paged_tensor_kernel<TQ4>);
    if (e != cudaSuccess) return e;
    using R = Regs<TQ4>;
    if (fa.numRegs != R::kLaunch) return cudaErrorInvalidConfiguration;
    CUtensorMap map{};
    if (!TQ4 && p.n_pages > 0 && (e = pool_map(p, &map)) != cudaSuccess) return e;
    e = cudaFuncSetAttribute(paged_tensor_kernel<TQ4>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemUsed);
    if (e != cudaSuccess) return e;
    // Launched while its predecessor runs, the kernel is there sooner (8 sequences of 4096
    // rows 27.1 us in a replayed graph, 28.2 else) but then runs 6% slower, for a reason not
    // known (512 tokens on 32,768 rows 3.41 ms, 3.2 else): for short calls, of at most some
    // 60 us, by the most steps that a pair can have.  The table's width bounds those, so a
    // table kept wide for the longest context is launched the other way.
    const int64_t tiles = p.max_tok * p.n_heads / kVecs + min(p.max_tok, (int64_t)p.n_seq);
    const int64_t rows = (int64_t)min(p.table_stride, p.n_pages) << p.shift;
    if (tiles * (rows / kRows + 1) <= 32 * kPagedPairs)
        return launch_chained(paged_tensor_kernel<TQ4>, 2 * kPagedPairs, kThreads, kSmemUsed, stream, p, map);
    paged_tensor_kernel<TQ4><<<2 * kPagedPairs, kThreads, kSmemUsed, stream>>>(p, map);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_tensor(kvq_format fmt, const PagedParams& p, cudaStream_t stream) {
    return fmt == KVQ_TQ4 ? launch<true>(p, stream) : launch<false>(p, stream);
}

}  // namespace kvq
