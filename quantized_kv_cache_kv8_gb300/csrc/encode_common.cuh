// encode_common.cuh -- the row encoders that the paged append shares with the row
// encoder kernels, fed from rotated rows in shared memory: TQ4 blocks (both use this
// one) and KV8 rows (kv8_encode_row_warp for any source).
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

// kv8_encode_row_warp with load(i) for element i of the row: the same bytes, the same
// error for a NaN or an infinity.
template <class Load>
__device__ __forceinline__ void kv8_encode_row_from(Load load, int n_blocks, int bd0, int bd1, uint8_t* cr, float* sr,
                                                    int lane, int32_t* err) {
    int off = 0;
    bool bad = false;
    for (int b = 0; b < n_blocks; ++b) {
        const int n = b == 0 ? bd0 : bd1;
        float amax = 0.0f;
        for (int i = lane; i < n; i += 32) {
            const float a = fabsf(load(off + i));
            bad |= !(a <= 3.402823466e38f);
            amax = fmaxf(amax, a);
        }
        amax = warp_max(amax);
        const float s = __fdiv_rn(amax, 448.0f);
        if (lane == 0) sr[b] = s;
        for (int i = lane; i < n; i += 32)
            cr[off + i] =
                s == 0.0f ? 0 : (uint8_t)__nv_cvt_float_to_fp8(__fdiv_rn(load(off + i), s), __NV_SATFINITE, __NV_E4M3);
        off += n;
    }
    if (__any_sync(kFull, bad) && lane == 0 && err) atomicCAS(err, 0, (int32_t)KVQ_ERR_NONFINITE);
}

struct Tq4Params {
    int32_t D, n_blocks, bd[2];
    float kn[2];      // (float)(1/sqrt(n)) per block
    float sqrtn[2];   // sqrtf((float)n) per block
    SignWords signs;
    Codebook16 cb;
};

// One scale block of N dims by one warp; load(i) gives element i of the block.
template <int N, class Load>
__device__ __forceinline__ void tq4_encode_block(Load load, int lane, const Tq4Params& p, int blk, const float* th,
                                                 uint8_t* __restrict__ out, float* scale_out, int32_t* err) {
    constexpr int K = N >= 32 ? N / 32 : 1;
    const bool active = (N >= 32) || (lane < N);
    float x[K], v[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = lane + 32 * k;
        x[k] = active ? load(i) : 0.0f;
        v[k] = (active && sign_neg(p.signs, blk, i)) ? -x[k] : x[k];
    }
    // sum of squares: per-lane fma chain over ascending elements, then halving
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) ss = __fmaf_rn(x[k], x[k], ss);
    ss = warp_sum(ss);
    // a NaN or infinite input, or a radius past the f32 range: no code exists
    if (!(ss <= 3.402823466e38f) && lane == 0 && err) atomicCAS(err, 0, (int32_t)KVQ_ERR_NONFINITE);
    const float s = __fdiv_rn(__fsqrt_rn(ss), p.sqrtn[blk]);
    warp_fwht<N>(v, lane);
    const float kn = p.kn[blk];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        int c = 0;
        if (s != 0.0f) c = code16(__fdiv_rn(__fmul_rn(v[k], kn), s), th);
        const int hi = __shfl_down_sync(kFull, c, 1);
        if (active && (lane & 1) == 0) out[(lane + 32 * k) >> 1] = (uint8_t)(c | (hi << 4));
    }
    if (lane == 0) *scale_out = s;
}

Tq4Params make_tq4_params(const kvq_mla_layout& L);

#define KVQ_POW2_CASES(MACRO) \
    MACRO(2) MACRO(4) MACRO(8) MACRO(16) MACRO(32) MACRO(64) MACRO(128) MACRO(256) MACRO(512) MACRO(1024)

}  // namespace kvq
