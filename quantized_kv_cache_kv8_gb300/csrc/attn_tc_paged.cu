// attn_tc_paged.cu -- tensor-core attention of new tokens over paged KV8 or TQ4
// rows, bf16 queries.
//
// A CTA walks over segments (paged_common.cuh): 64 query vectors -- consecutive
// (token, head) pairs of one sequence, whatever the head count -- against a run
// of 128-row steps.  Both products are transposed, rows (or dims) on M = 128 and
// the 64 vectors on N:
//   S^T = C Q^T   (A = codes, K-major; the latent and the rope dims into an
//                  accumulator each, as each has its own row scale)
//   O^T += C^T P^T (A = the same codes read MN-major, 4 blocks of 128 dims)
// because 64 x 512 f32 of context is half of tensor memory and M = 64 forms run
// at half rate.  A step's rows are decoded once to f16 (e4m3 codes exactly, the
// 16 levels of TQ4 times kGamma within 9.3e-5) into nine 64-dim chunks of
// swizzled shared memory (144 KB), next to the queries (72 KB).
//
// A bf16 query vector times a power of two of its own is exact in f16 (down to
// 2^-24 of 2^14); the rotated query of TQ4 is rounded once, 2^-12 relative.
//
// Step t: 16 worker warps store the step's codes chunk group by chunk group
// (dims 0-255, 256-511, rope) as the context products of step t-1 release the
// chunks; a 17th warp issues score products group by group behind
// them, and the context products once the weights are written.  The next step's
// codes are on their way to registers before the softmax.  16 warps, because a
// step is a chain (store, score, softmax, context) and its links are as long as
// a warp's share of them.
//
// Softmax, per query vector, in log2 units: m is a lagged running maximum of the
// scores, p = 2^(z - m) enters the row sum in f32, and the context takes the f16
// weight w = p s_L E, E = 2^(m - R - 3) with R the largest z + log2 s_L of the
// steps that set the references, so that weights are relative to the largest
// p s_L and rows of small latent scale keep f16 precision where they matter.  A
// score that passes m by more than 2^14, or a latent scale past 3.5 / max E,
// sends the step down the exact path: column maxima, new m, R and E, O^T
// rescaled in tensor memory.  Both limits keep w under the f16 maximum.
// Rows that a vector does not see (causal end, vectors of shorter limits) get
// z = -inf; a vector that has seen no row has m = -inf and E = 0.
#include "tc_common.cuh"
#include "paged_common.cuh"

#include <math.h>

namespace kvq {
namespace {
using namespace tc;

constexpr int kRows = PagedTensor::kN;      // rows a step
constexpr int kCols = PagedTensor::kM;      // query vectors
constexpr int kWarps = 16;                  // worker warps
constexpr int kWorkers = 32 * kWarps;
constexpr int kThreads = kWorkers + 64;     // ... and the issuing and the walking warp: 112 registers a thread
constexpr int kChunks = 9, kRope = 8;       // the rope chunk's slot holds P^T after the score
constexpr uint32_t kSlotBytes = kRows * 128, kQChunkBytes = kCols * 128;
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffSlot = kOffQ + kChunks * kQChunkBytes;
constexpr uint32_t kOffM = kOffSlot + kChunks * kSlotBytes;
constexpr uint32_t kOffR = kOffM + kCols * 4;
constexpr uint32_t kOffE = kOffR + kCols * 4;
constexpr uint32_t kOffF = kOffE + kCols * 4;          // 1 / E
constexpr uint32_t kOffCz = kOffF + kCols * 4;         // score scale of a vector (sm log2 e / its query scale)
constexpr uint32_t kOffAlpha = kOffCz + kCols * 4;     // O^T rescale; row sums and output factors at the end
constexpr uint32_t kOffAlphaM = kOffAlpha + kCols * 4; // row-sum rescale
constexpr uint32_t kOffLim = kOffAlphaM + kCols * 4;   // rows each vector sees
constexpr uint32_t kOffRow = kOffLim + kCols * 4;      // pool rows of two steps
constexpr uint32_t kOffRed = kOffRow + 2 * kRows * 4;  // 2 x 4 quadrants x 64 vectors
constexpr uint32_t kOffBar = kOffRed + 2 * 4 * kCols * 4;
constexpr uint32_t kOffLevels = kOffBar + 16 * 8;      // f16 levels as byte planes
constexpr uint32_t kOffEmax = kOffLevels + 32;
constexpr uint32_t kOffMisc = kOffEmax + 16;           // abort flag, TMEM base
constexpr uint32_t kOffPart = kOffMisc + 16;           // scan of the work split
constexpr uint32_t kOffWork = kOffPart + (kThreads / 32 + 2) * 8;   // two segments, announced one ahead
constexpr uint32_t kSmemUsed = kOffWork + 2 * 64;
static_assert(kOffSlot % 1024 == 0 && kOffPart % 8 == 0, "alignment");
static_assert(kSmemUsed <= 232448, "shared memory budget");
constexpr int kStageStride = 516;           // floats between staged output vectors
static_assert(kCols * kStageStride * 4 <= kChunks * kSlotBytes, "output stage");

constexpr uint32_t kColO = 0, kColSL = 256, kColSR = 320, kTmemCols = 512;

// mbarriers: chunk group stored (16 warps), chunk pair released by the context
// products, scores complete, weights written (16 warps), all products complete,
// one that nothing arrives on (the testing hook's stall), segment announced,
// segment done with (16 warps and the issuing thread)
enum {
    kBarFull0 = 0, kBarFree0 = 3, kBarScore = 7, kBarP = 8, kBarDone = 9, kBarNever = 10, kBarWork0 = 11,
    kBarWorkFree0 = 13, kNumBars = 15
};

// A segment as the workers use it; steps = 0 ends the walk.
struct Work {
    int32_t steps, b, rows;
    int32_t first, end, seen0;   // first row; rows that some vector sees; rows that the first one sees
    int64_t row0, tok0, base, slot, parts;
};
static_assert(sizeof(Work) <= 64, "segment record");

constexpr float kLagLog2 = 14.0f, kScaleLim = 3.5f, kHeadroom = 3.0f, kLogEmax = 120.0f;
// levels times this round to f16 within 9.3e-5 (unscaled: 3.2e-4); divided out in f32
constexpr float kGamma = 1.3338516f;
constexpr uint32_t kIdescScore = idesc_f16(128, kCols, false, false);
constexpr uint32_t kIdescCtx = idesc_f16(128, kCols, true, true);

// ---- a worker's raw share of a step -------------------------------------------
// KV8, groups of 256 bytes a row: 4 pieces of 16 bytes, piece i at row
// 2 (warp + 16 i) + (lane / 4) % 2, bytes 64 (lane / 8) + 16 (lane % 4): a warp
// reads two whole runs of 256 bytes, and the 8 lanes that a shared store serves
// at a time write one chunk of two adjacent rows, 8 different 16-byte units.
// Rope: one piece, row tid / 4, bytes 16 (tid % 4).
// TQ4, groups of 128 bytes a row: 2 pieces, piece i at row 8 warp + lane % 8,
// bytes 64 i + 16 (lane / 8): 8 lanes store one unit of 8 rows, whose swizzle
// phases differ.  Rope (32 bytes): warps 0-7, row 16 warp + lane % 8 +
// 8 (lane / 16), bytes 16 ((lane / 8) % 2).
template <bool TQ4>
struct Raw {
    static constexpr int kPer = TQ4 ? 2 : 4;
    uint4 a[kPer], b[kPer], c;
};
template <bool TQ4>
__device__ __forceinline__ int piece_row(int i, int warp, int lane) {
    return TQ4 ? 8 * warp + (lane & 7) : 2 * (warp + 16 * i) + ((lane >> 2) & 1);
}
template <bool TQ4>
__device__ __forceinline__ int piece_byte(int i, int lane) {
    return TQ4 ? 64 * i + 16 * (lane >> 3) : 64 * (lane >> 3) + 16 * (lane & 3);
}
template <bool TQ4>
__device__ __forceinline__ int rope_row(int tid, int warp, int lane) {
    return TQ4 ? 16 * warp + (lane & 7) + 8 * (lane >> 4) : tid >> 2;
}
template <bool TQ4>
__device__ __forceinline__ int rope_byte(int tid, int lane) {
    return TQ4 ? 16 * ((lane >> 3) & 1) : 16 * (tid & 3);
}
template <bool TQ4>
__device__ __forceinline__ void load_raw(Raw<TQ4>& r, const uint8_t* __restrict__ codes, const int32_t* prow, int nt,
                                         int tid, int warp, int lane) {
    constexpr int kRow = TQ4 ? kMlaD / 2 : kMlaD, kGroup = TQ4 ? 128 : 256;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < Raw<TQ4>::kPer; ++i) {
        const int row = piece_row<TQ4>(i, warp, lane);
        const uint8_t* src = codes + (int64_t)prow[row] * kRow + piece_byte<TQ4>(i, lane);
        r.a[i] = row < nt ? __ldg(reinterpret_cast<const uint4*>(src)) : z;
        r.b[i] = row < nt ? __ldg(reinterpret_cast<const uint4*>(src + kGroup)) : z;
    }
    r.c = z;
    if (!TQ4 || warp < 8) {
        const int row = rope_row<TQ4>(tid, warp, lane);
        if (row < nt)
            r.c = __ldg(reinterpret_cast<const uint4*>(codes + (int64_t)prow[row] * kRow + 2 * kGroup +
                                                       rope_byte<TQ4>(tid, lane)));
    }
}

// 16 e4m3 codes -> 16 f16 at byte offset b of swizzled row `row`.
__device__ __forceinline__ void store_kv8(unsigned char* slot, const uint4& c, int row, int b) {
    const uint32_t in[4] = {c.x, c.y, c.z, c.w};
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) e4m3x4_to_half2x2(in[i], w[2 * i], w[2 * i + 1]);
    *reinterpret_cast<uint4*>(slot + sw128(row, b)) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(slot + sw128(row, b + 16)) = make_uint4(w[4], w[5], w[6], w[7]);
}
// 32 nibble codes -> 32 f16 levels (64 bytes) by byte permutes over the low and
// the high bytes of the levels: the low 3 bits of a code pick among levels 0-7
// and 8-15, bit 3 between the two.
struct Planes {
    uint32_t lo[4], hi[4];
};
__device__ __forceinline__ void store_tq4(unsigned char* slot, const uint4& c, int row, int b, const Planes& t) {
    const uint32_t in[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t sel = in[i] & 0x77777777u, pick = ((in[i] >> 1) & 0x44444444u) | 0x32103210u;
        uint32_t w[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t s = h ? sel >> 16 : sel, k = h ? pick >> 16 : pick;
            const uint32_t lo = __byte_perm(__byte_perm(t.lo[0], t.lo[1], s), __byte_perm(t.lo[2], t.lo[3], s), k);
            const uint32_t hi = __byte_perm(__byte_perm(t.hi[0], t.hi[1], s), __byte_perm(t.hi[2], t.hi[3], s), k);
            w[2 * h] = __byte_perm(lo, hi, 0x5140u);
            w[2 * h + 1] = __byte_perm(lo, hi, 0x7362u);
        }
        *reinterpret_cast<uint4*>(slot + sw128(row, b + 16 * i)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
template <bool TQ4>
__device__ __forceinline__ void store_group(unsigned char* sSlot, const uint4 (&v)[Raw<TQ4>::kPer], int g, int warp,
                                            int lane, const Planes& t) {
#pragma unroll
    for (int i = 0; i < Raw<TQ4>::kPer; ++i) {
        const int row = piece_row<TQ4>(i, warp, lane), byte = piece_byte<TQ4>(i, lane);
        if (TQ4) store_tq4(sSlot + (4 * g + (byte >> 5)) * kSlotBytes, v[i], row, 4 * (byte & 31), t);
        else store_kv8(sSlot + (4 * g + (byte >> 6)) * kSlotBytes, v[i], row, 2 * (byte & 63));
    }
}

// One MMA, or one commit, of a whole warp in step: the warp computes the
// descriptors together (in uniform registers) and one elected lane, always the
// same, issues.  A lone lane in a branch of its own spends about 115 cycles an
// MMA on moving its operands; this way N = 64 runs at the 48 cycles that its 6 KB
// of operands take to read.
__device__ __forceinline__ void umma_one(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void commit_one(uint64_t* bar) {
    asm volatile(
        "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, long long limit) {
    return __all_sync(kFull, mbar_wait(bar, parity, abort_flag, limit));
}

__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// ---- queries ------------------------------------------------------------------
// Four vectors a warp: to f16 under a power of two that puts the largest element
// in [2^13, 2^14); sCz gets what undoes it in the score.
template <bool TQ4>
__device__ __forceinline__ void load_queries(const PagedParams& p, const Work& g, unsigned char* sQ, float* sCz,
                                             int warp, int lane) {
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
#pragma unroll 1
    for (int k = 0; k < kCols / kWarps; ++k) {
        const int r = (kCols / kWarps) * warp + k;
        float v[18];
        const int64_t at = (g.row0 + r) * kMlaD;
        if (TQ4) {
            // element lane + 32 i
#pragma unroll
            for (int i = 0; i < 18; ++i) v[i] = r < g.rows ? __bfloat162float(q[at + lane + 32 * i]) : 0.0f;
            float rot[16], rope[2];
#pragma unroll
            for (int i = 0; i < 16; ++i) rot[i] = sign_neg(p.signs, 0, lane + 32 * i) ? -v[i] : v[i];
            warp_fwht<512>(rot, lane);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = rot[i] * p.kn[0];
#pragma unroll
            for (int i = 0; i < 2; ++i) rope[i] = sign_neg(p.signs, 1, lane + 32 * i) ? -v[16 + i] : v[16 + i];
            warp_fwht<64>(rope, lane);
#pragma unroll
            for (int i = 0; i < 2; ++i) v[16 + i] = rope[i] * p.kn[1];
        } else {
            // elements 2 (lane + 32 i), + 1
            const uint32_t* qw = reinterpret_cast<const uint32_t*>(q + at);
#pragma unroll
            for (int i = 0; i < 9; ++i) {
                const uint32_t w = r < g.rows ? __ldg(qw + lane + 32 * i) : 0u;
                v[2 * i] = __uint_as_float(w << 16);
                v[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
            }
        }
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 18; ++i) top = fmaxf(top, fabsf(v[i]));
        top = warp_max(top);
        int e = 14;
        if (top > 0.0f && top <= 3.402823466e38f) frexpf(top, &e);
        e = max(e, -100);   // 2^(14 - e) stays finite
        const float scale = ldexpf(1.0f, 14 - e);
        if (lane == 0) sCz[r] = p.sm_scale * kLog2e * ldexpf(1.0f, e - 14) * (TQ4 ? 1.0f / kGamma : 1.0f);
        if (TQ4) {
#pragma unroll
            for (int i = 0; i < 18; ++i) {
                const int d = lane + 32 * i;
                *reinterpret_cast<__half*>(sQ + (d >> 6) * kQChunkBytes + sw128(r, (d & 63) * 2)) =
                    __float2half_rn(v[i] * scale);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 9; ++i)
                *reinterpret_cast<__half2*>(sQ + i * kQChunkBytes + sw128(r, lane * 4)) =
                    __floats2half2_rn(v[2 * i] * scale, v[2 * i + 1] * scale);
        }
    }
}

// One thread's row of scores: 16 vectors, d = z - m (sub = their m) or z itself.
struct RowView {
    uint32_t tmem;     // lane base + first column of the 16
    float sl, sr;      // row scales
    int32_t t;         // row within the sequence
    bool ok, mask;     // row within the step; some vector of the tile does not see the step's end
};
__device__ __forceinline__ void load_scores(const RowView& v, const float* cz, const float* sub, const int32_t* lim,
                                            float (&z)[16]) {
    uint32_t l[16], r[16];
    tmem_ld16(v.tmem + kColSR, r);
    tmem_ld16(v.tmem + kColSL, l);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 c = *reinterpret_cast<const float4*>(cz + 4 * i);
        const float4 m = sub ? *reinterpret_cast<const float4*>(sub + 4 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float cv[4] = {c.x, c.y, c.z, c.w}, mv[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int j = 4 * i + k;
            const float s = fmaf(__uint_as_float(l[j]), v.sl, __uint_as_float(r[j]) * v.sr);
            z[j] = v.ok ? fmaf(s, cv[k], -mv[k]) : -INFINITY;
        }
    }
    if (v.mask) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (v.t >= lim[j]) z[j] = -INFINITY;
    }
}

// The exact path of a step, by every worker (out of line: rare).
__device__ __noinline__ void exact_path(unsigned char* sm, uint32_t tmem, RowView view, int hq, int lane, int warp,
                                        int tid, bool first, uint32_t* exact_count) {
    float* sM = reinterpret_cast<float*>(sm + kOffM);
    float* sR = reinterpret_cast<float*>(sm + kOffR);
    float* sAlpha = reinterpret_cast<float*>(sm + kOffAlpha);
    float* sRed = reinterpret_cast<float*>(sm + kOffRed);
    const float* cz = reinterpret_cast<const float*>(sm + kOffCz) + 16 * hq;
    const int32_t* lim = reinterpret_cast<const int32_t*>(sm + kOffLim) + 16 * hq;
    {
        float z[16];
        const int at = (warp & 3) * kCols + 16 * hq + (lane & 15);
        load_scores(view, cz, nullptr, lim, z);
        float top = warp_columns16<true>(z, lane);
        if (lane < 16) sRed[at] = top;
        load_scores(view, cz, nullptr, lim, z);
        const float add = view.sl > 0.0f ? __log2f(view.sl) : -INFINITY;   // -inf: an inert latent block
#pragma unroll
        for (int j = 0; j < 16; ++j) z[j] += add;
        top = warp_columns16<true>(z, lane);
        if (lane < 16) sRed[4 * kCols + at] = top;
    }
    worker_sync<kWorkers>();
    if (tid < kCols) {
        const float* ry = sRed + 4 * kCols;
        const float c4 = fmaxf(fmaxf(sRed[tid], sRed[kCols + tid]), fmaxf(sRed[2 * kCols + tid], sRed[3 * kCols + tid]));
        const float y4 = fmaxf(fmaxf(ry[tid], ry[kCols + tid]), fmaxf(ry[2 * kCols + tid], ry[3 * kCols + tid]));
        const float mo = sM[tid], mn = fmaxf(mo, c4);
        const float ro = sR[tid], rn = fmaxf(ro, y4);
        const float dn = fminf(mn - rn - kHeadroom, kLogEmax), d_old = fminf(mo - ro - kHeadroom, kLogEmax);
        reinterpret_cast<float*>(sm + kOffAlphaM)[tid] = mo == -INFINITY ? 0.0f : ex2(mo - mn);
        // O^T holds sum p s_L E c: rescaled by (E_new / E_old) 2^(m_old - m_new)
        sAlpha[tid] = ro == -INFINITY ? 0.0f : ex2(dn - d_old + (mo - mn));
        sM[tid] = mn;
        sR[tid] = rn;
        // no latent scale met yet: E = 0, and the next one takes this path (max E
        // infinite); no row seen at all: the first score takes it by m = -inf
        const bool none = rn == -INFINITY;
        const float e = none ? 0.0f : ex2(dn);
        reinterpret_cast<float*>(sm + kOffE)[tid] = e;
        reinterpret_cast<float*>(sm + kOffF)[tid] = none ? 0.0f : ex2(-dn);
        const float em = warp_max(mn == -INFINITY ? 0.0f : none ? INFINITY : e);
        if (lane == 0) reinterpret_cast<float*>(sm + kOffEmax)[tid >> 5] = em;
        if (!first && tid == 0) atomicAdd(exact_count, 1u);
    }
    worker_sync<kWorkers>();
    if (!first) {
        // every context product so far is complete: the score commit of this
        // step follows them
        const uint32_t ta = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kColO + 64 * hq;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            uint32_t o[16];
            tmem_ld16(ta + 16 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * sAlpha[16 * c + j]);
            tmem_st16(ta + 16 * c, o);
        }
        tmem_wait_st();
    }
}

template <bool TQ4>
__global__ void __launch_bounds__(kThreads, 1) paged_tensor_kernel(const __grid_constant__ PagedParams p) {
    launch_dependents();
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* sm = smem_raw;
    unsigned char* sQ = sm + kOffQ;
    unsigned char* sSlot = sm + kOffSlot;
    unsigned char* sP = sSlot + kRope * kSlotBytes;
    float* sM = reinterpret_cast<float*>(sm + kOffM);
    float* sR = reinterpret_cast<float*>(sm + kOffR);
    float* sE = reinterpret_cast<float*>(sm + kOffE);
    float* sF = reinterpret_cast<float*>(sm + kOffF);
    float* sCz = reinterpret_cast<float*>(sm + kOffCz);
    float* sAlpha = reinterpret_cast<float*>(sm + kOffAlpha);
    float* sAlphaM = reinterpret_cast<float*>(sm + kOffAlphaM);
    int32_t* sLim = reinterpret_cast<int32_t*>(sm + kOffLim);
    int32_t* sRow = reinterpret_cast<int32_t*>(sm + kOffRow);
    float* sRed = reinterpret_cast<float*>(sm + kOffRed);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kOffBar);
    unsigned char* sLevels = sm + kOffLevels;
    float* sEmax = reinterpret_cast<float*>(sm + kOffEmax);
    volatile int* sAbort = reinterpret_cast<volatile int*>(sm + kOffMisc);
    uint32_t* sTmem = reinterpret_cast<uint32_t*>(sm + kOffMisc + 4);
    int64_t* sPart = reinterpret_cast<int64_t*>(sm + kOffPart);
    Work* sWork = reinterpret_cast<Work*>(sm + kOffWork);

    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFull, tid >> 5, 0);
    const int64_t cta = blockIdx.x;
    const int64_t wl = p.wait_limit;
    if (tid < 4) p.ws_desc[cta * 4 + tid] = 0;
    PagedWalk<PagedTensor> walk;
    if (!walk.template start<kThreads>(p, cta, gridDim.x, sPart)) return;
    if (smem_u32(smem_raw) & 1023u) {   // the swizzled operands would be misread
        if (tid == 0) set_err(p.err, KVQ_ERR_DEVICE);
        return;
    }

    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(sTmem)),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid == 64) {
        for (int i = 0; i < kNumBars; ++i) {
            const uint32_t count = (i < kBarFree0 || i == kBarP) ? (uint32_t)kWarps
                                   : i >= kBarWorkFree0          ? (uint32_t)kWarps + 1u
                                                                 : 1u;
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(&bars[i])), "r"(count));
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *sAbort = 0;
    }
    if (TQ4 && tid == 0) {
        uint32_t lo[4] = {0u, 0u, 0u, 0u}, hi[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const uint32_t h = __half_as_ushort(__float2half_rn(__fmul_rn(p.lv[k], kGamma)));
            lo[k >> 2] |= (h & 0xffu) << (8 * (k & 3));
            hi[k >> 2] |= (h >> 8) << (8 * (k & 3));
        }
        *reinterpret_cast<uint4*>(sLevels) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        *reinterpret_cast<uint4*>(sLevels + 16) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = *sTmem;

    if (warp >= kWarps) {
        // ================= the walk: announces segments one ahead =================
        if (warp == kWarps + 1 && lane == 0) {
            bool more = true;
            for (int n = 0; more; ++n, walk.next(p)) {
                if (n >= 2 && !mbar_wait(&bars[kBarWorkFree0 + (n & 1)], (uint32_t)(n / 2 - 1) & 1u, sAbort, wl)) break;
                Segment g;
                Work w{};
                more = walk.get(p, g);
                if (more) {
                    w.steps = (int32_t)(g.u1 - g.u0);
                    w.b = g.b;
                    w.rows = g.rows;
                    w.first = (int32_t)(g.u0 * kRows);
                    w.end = (int32_t)row_limit(g, g.rows - 1, p.n_heads);
                    w.seen0 = (int32_t)row_limit(g, 0, p.n_heads);
                    w.row0 = g.row0;
                    w.tok0 = g.tok0;
                    w.base = g.base;
                    w.slot = walk.slot(g, cta, &w.parts);
                }
                sWork[n & 1] = w;
                mbar_arrive(&bars[kBarWork0 + (n & 1)]);
            }
        }
        // ================= the issuing warp =================
        if (warp == kWarps) {
            const uint64_t dq0 = umma_desc(smem_u32(sQ), 16, 1024);
            const uint64_t dslot0 = umma_desc(smem_u32(sSlot), 16, 1024);
            const uint64_t dpair0 = umma_desc(smem_u32(sSlot), kSlotBytes, 1024);
            const uint64_t dp = umma_desc(smem_u32(sP), kSlotBytes, 1024);
            constexpr uint64_t kQStep = kQChunkBytes >> 4, kSlotStep = kSlotBytes >> 4;
            bool ok = true;
            if (p.stall_polls > 0) ok = warp_wait(&bars[kBarNever], 0u, sAbort, p.stall_polls);
            uint32_t it = 0;
            for (int n = 0; ok; ++n) {
                ok = warp_wait(&bars[kBarWork0 + (n & 1)], (uint32_t)(n >> 1) & 1u, sAbort, wl);
                if (!ok) break;
                const int steps = __shfl_sync(kFull, sWork[n & 1].steps, 0);
                if (steps == 0) break;
                warp_arrive(&bars[kBarWorkFree0 + (n & 1)], lane);
                for (int t = 0; t < steps && ok; ++t, ++it) {
                    const uint32_t par = it & 1u;
#pragma unroll
                    for (int gr = 0; gr < 3; ++gr) {
                        ok = ok && warp_wait(&bars[kBarFull0 + gr], par, sAbort, wl);
                        if (!ok) break;
                        tc_after();
#pragma unroll
                        for (int kc = 4 * gr; kc < (gr < 2 ? 4 * gr + 4 : kChunks); ++kc)
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                umma_one(tmem + (kc < kRope ? kColSL : kColSR), dslot0 + kc * kSlotStep + 2 * ks,
                                         dq0 + kc * kQStep + 2 * ks, kIdescScore,
                                         ((kc == 0 || kc == kRope) && ks == 0) ? 0u : 1u);
                    }
                    commit_one(&bars[kBarScore]);
                    ok = ok && warp_wait(&bars[kBarP], par, sAbort, wl);
                    if (!ok) break;
                    tc_after();
#pragma unroll
                    for (int db = 0; db < 4; ++db) {
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            umma_one(tmem + kColO + 64 * db, dpair0 + 2 * db * kSlotStep + 128 * ks, dp + 128 * ks,
                                     kIdescCtx, (t > 0 || ks > 0) ? 1u : 0u);
                        commit_one(&bars[kBarFree0 + db]);
                    }
                }
            }
            commit_one(&bars[kBarDone]);
        }
        return;
    }

    // ================= workers =================
    const int srow = 32 * (warp & 3) + lane;   // softmax: this thread's row (TMEM lane)
    const int hq = warp >> 2;                   // ... and vectors 16 hq .. 16 hq + 15
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    uint32_t it = 0;
    bool aborted = false;
    for (int n = 0;; ++n) {
        if (!mbar_wait(&bars[kBarWork0 + (n & 1)], (uint32_t)(n >> 1) & 1u, sAbort, wl)) aborted = true;
        if (worker_any<kWorkers>(aborted)) {
            aborted = true;
            break;
        }
        const Work& g = sWork[n & 1];
        const int steps = g.steps;
        if (steps == 0) break;
        // ---- prologue: state, limits, queries, the first step's rows ----
        const int32_t first = g.first, end = g.end;
        // a row of step t (tid < kRows): its page is asked for early, and turned
        // into a pool row where it is stored; rows past the end get row 0, never read
        const int32_t* table = p.table + (int64_t)g.b * p.table_stride;
        auto page_of = [&](int t) -> int32_t {
            const int32_t r = first + t * kRows + tid;
            return (tid < kRows && t < steps && r < end) ? __ldg(table + (r >> p.shift)) : 0;
        };
        auto set_row = [&](int t, int32_t id) {
            if (tid >= kRows) return;
            if (id < 0 || id >= p.n_pages) {
                set_err(p.err, KVQ_ERR_ARG);
                id = 0;
            }
            const int32_t r = first + t * kRows + tid;
            sRow[(t & 1) * kRows + tid] = (id << p.shift) + (r & ((1 << p.shift) - 1));
        };
        auto rows_in = [&](int t) { return max(0, min(kRows, end - first - t * kRows)); };
        {
            const int32_t id0 = page_of(0), id1 = page_of(1);
            set_row(0, id0);
            set_row(1, id1);
        }
        if (tid < kCols) {
            sM[tid] = -INFINITY;
            sR[tid] = -INFINITY;
            sE[tid] = 0.0f;
            sF[tid] = 0.0f;
            // vectors past the tile's last repeat its limit: they score 0 and are dropped
            sLim[tid] = (int32_t)max((int64_t)0, g.base + 1 + (g.tok0 + min(tid, g.rows - 1)) / p.n_heads);
            if (tid < kCols / 32) sEmax[tid] = 0.0f;
        }
        load_queries<TQ4>(p, g, sQ, sCz, warp, lane);
        fence_async_smem();
        worker_sync<kWorkers>();
        float lsum[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) lsum[j] = 0.0f;
        Raw<TQ4> raw;
        float sl_next = 0.0f, sr_next = 0.0f;
        auto request = [&](int t) {   // codes and scales of step t
            const int32_t* rows = sRow + (t & 1) * kRows;
            const int nt = rows_in(t);
            load_raw<TQ4>(raw, p.codes, rows, nt, tid, warp, lane);
            sl_next = sr_next = 0.0f;
            if (srow < nt) {
                const float* s = p.scales + (int64_t)rows[srow] * p.n_blocks;
                sl_next = s[0];
                sr_next = s[p.n_blocks - 1];
            }
        };
        request(0);
        int t = 0;
        for (; t < steps; ++t, ++it) {
            const uint32_t par = it & 1u, prev = par ^ 1u;
            const int32_t page2 = page_of(t + 2);
            const RowView view{tmem + lane_base + 16 * hq, sl_next, sr_next, first + t * kRows + srow,
                               srow < rows_in(t), first + (t + 1) * kRows > g.seen0};
            // ---- decode: dims 0-255, 256-511, rope ----
            {
                Planes pl;
                if (TQ4) {
                    const uint4 a = *reinterpret_cast<const uint4*>(sLevels), b = *reinterpret_cast<const uint4*>(sLevels + 16);
                    pl = Planes{{a.x, a.y, a.z, a.w}, {b.x, b.y, b.z, b.w}};
                }
#pragma unroll
                for (int gr = 0; gr < 2; ++gr) {
                    if (it > 0) {
                        mbar_wait(&bars[kBarFree0 + 2 * gr], prev, sAbort, wl);
                        mbar_wait(&bars[kBarFree0 + 2 * gr + 1], prev, sAbort, wl);
                    }
                    store_group<TQ4>(sSlot, gr == 0 ? raw.a : raw.b, gr, warp, lane, pl);
                    fence_async_smem();
                    warp_arrive(&bars[kBarFull0 + gr], lane);
                }
                if (!TQ4) store_kv8(sP, raw.c, rope_row<TQ4>(tid, warp, lane), 2 * rope_byte<TQ4>(tid, lane));
                else if (warp < 8) store_tq4(sP, raw.c, rope_row<TQ4>(tid, warp, lane), 4 * rope_byte<TQ4>(tid, lane), pl);
                fence_async_smem();
                warp_arrive(&bars[kBarFull0 + 2], lane);
            }
            if (t + 1 < steps) request(t + 1);

            // ---- softmax: one warp polls, the others wait on the named barrier ----
            if (warp == 1) mbar_wait(&bars[kBarScore], par, sAbort, wl);
            worker_sync<kWorkers>();
            tc_after();
            set_row(t + 2, page2);   // step t's rows are no longer needed
            float z[16];
            load_scores(view, sCz + 16 * hq, sM + 16 * hq, sLim + 16 * hq, z);
            float dmax = z[0];
#pragma unroll
            for (int j = 1; j < 16; ++j) dmax = fmaxf(dmax, z[j]);
            const float emax = fmaxf(sEmax[0], sEmax[1]);
            const bool flag = (*sAbort != 0) | (view.sl * emax > kScaleLim) | (dmax > kLagLog2);
            if (worker_any<kWorkers>(flag)) {
                if (worker_any<kWorkers>(*sAbort != 0)) {
                    aborted = true;
                    break;
                }
                exact_path(sm, tmem, view, hq, lane, warp, tid, t == 0, p.exact_count);
#pragma unroll
                for (int j = 0; j < 16; ++j) lsum[j] *= sAlphaM[16 * hq + j];
                load_scores(view, sCz + 16 * hq, sM + 16 * hq, sLim + 16 * hq, z);
            }
            {
                uint32_t pk[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 e = *reinterpret_cast<const float4*>(sE + 16 * hq + 4 * i);
                    const float ev[4] = {e.x * view.sl, e.y * view.sl, e.z * view.sl, e.w * view.sl};
#pragma unroll
                    for (int k = 0; k < 4; k += 2) {
                        const int j = 4 * i + k;
                        z[j] = ex2(z[j]);
                        z[j + 1] = ex2(z[j + 1]);
                        const __half2 h2 = __floats2half2_rn(z[j] * ev[k], z[j + 1] * ev[k + 1]);
                        pk[j / 2] = *reinterpret_cast<const uint32_t*>(&h2);
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<uint4*>(sP + sw128(srow, 32 * hq + 16 * i)) =
                        make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
            }
            fence_async_smem();
            tc_before();
            warp_arrive(&bars[kBarP], lane);
#pragma unroll
            for (int j = 0; j < 16; ++j) lsum[j] += z[j];
        }
        if (aborted) break;

        // ---- epilogue: the last context products, row sums, O^T out ----
        if (!mbar_wait(&bars[kBarFree0 + 3], (it - 1) & 1u, sAbort, wl)) aborted = true;
        tc_after();
        if (worker_any<kWorkers>(aborted)) {
            aborted = true;
            break;
        }
        {
            const float s = warp_columns16<false>(lsum, lane);
            if (lane < 16) sRed[(warp & 3) * kCols + 16 * hq + lane] = s;
        }
        worker_sync<kWorkers>();
        const int64_t slot = g.slot;
        if (tid < kCols) {
            const float l = (sRed[tid] + sRed[kCols + tid]) + (sRed[2 * kCols + tid] + sRed[3 * kCols + tid]);
            const float f = TQ4 ? sF[tid] / kGamma : sF[tid];
            sAlpha[tid] = slot >= 0 ? f : (l == 0.0f ? 0.0f : f / l);   // no visible row: zeros
            if (slot >= 0) {
                float* ml = p.ws_ml + (slot * kCols + tid) * 2;
                ml[0] = sM[tid] * kLn2;
                ml[1] = l;
            }
        }
        if (g.parts > 0 && tid == 0) {
            p.ws_desc[cta * 4] = g.parts;
            p.ws_desc[cta * 4 + 1] = g.row0;
            p.ws_desc[cta * 4 + 2] = g.rows;
        }
        worker_sync<kWorkers>();
        const int dim = 128 * hq + 32 * (warp & 3) + lane;   // block hq of the context
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out);
        float* stage = reinterpret_cast<float*>(sSlot);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            uint32_t v[16];
            tmem_ld16(tmem + lane_base + kColO + 64 * hq + 16 * c, v);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int r = 16 * c + j;
                const float x = __uint_as_float(v[j]) * sAlpha[r];
                if (slot >= 0) p.ws_o[(slot * kCols + r) * kMlaDV + dim] = x;
                else if (TQ4) stage[r * kStageStride + dim] = x;
                else if (r < g.rows) out[(g.row0 + r) * kMlaDV + dim] = __float2bfloat16_rn(x);
            }
        }
        if (TQ4 && slot < 0) {
            worker_sync<kWorkers>();
            for (int r = warp; r < g.rows; r += kWarps) {
                float v[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = stage[r * kStageStride + lane + 32 * k];
                warp_fwht<512>(v, lane);
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const int i = lane + 32 * k;
                    const float y = v[k] * p.kn[0];
                    out[(g.row0 + r) * kMlaDV + i] = __float2bfloat16_rn(sign_neg(p.signs, 0, i) ? -y : y);
                }
            }
        }
        warp_arrive(&bars[kBarWorkFree0 + (n & 1)], lane);
        tc_before();
        worker_sync<kWorkers>();   // O^T, the stage and the state are free for the next segment
        tc_after();
    }
    {
        // bounded, and not cut short by the abort flag: TMEM is released only
        // after the products in flight have completed
        volatile int never = 0;
        if (!mbar_wait(&bars[kBarDone], 0u, &never)) aborted = true;
    }
    if (aborted && tid == 0) set_err(p.err, KVQ_ERR_TIMEOUT);
    tc_before();
    worker_sync<kWorkers>();
    tc_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
}

template <bool TQ4>
cudaError_t launch(const PagedParams& p, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(paged_tensor_kernel<TQ4>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemUsed);
    if (e != cudaSuccess) return e;
    paged_tensor_kernel<TQ4><<<kPagedCtas, kThreads, kSmemUsed, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_tensor(kvq_format fmt, const PagedParams& p, cudaStream_t stream) {
    return fmt == KVQ_TQ4 ? launch<true>(p, stream) : launch<false>(p, stream);
}

}  // namespace kvq
