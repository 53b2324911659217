// encode_common.cuh -- the TQ4 block encoder shared by the row encoder and the
// paged append, which feeds it rotated rows from shared memory.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

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
