// gqa.cuh -- launches of the grouped-query KV8 pools and of beam search, for the C
// entry points: append (gqa_append.cu), attention (gqa_attn.cu), selection (beam.cu),
// page sharing (fork.cu).
#pragma once

#include "paged.cuh"

namespace kvq {

struct GqaAttnCall {
    const void* q;
    kvq_dtype dtype;
    int64_t n_tokens;
    int32_t n_heads, n_kv_heads, head_dim, n_seq;
    const int64_t* cu_q;
    const uint8_t* k_codes;
    const uint8_t* v_codes;
    const float* scales;
    const int32_t* table;
    int32_t table_stride;
    const int64_t* kv_lens;
    int32_t page_rows, n_pages;
    float sm_scale;
    int32_t causal;
    void* out;
    void* workspace;
};
size_t gqa_attn_workspace_bytes(int32_t head_dim);
cudaError_t launch_gqa_attn(const GqaAttnCall& c, cudaStream_t stream);

struct GqaAppendCall {
    const kvq_rope* rope;   // null: no rotation
    kvq_dtype dtype;
    int64_t n;
    int32_t n_heads, n_kv_heads, head_dim;
    const void* k;
    int64_t k_token, k_head;
    const void* v;
    int64_t v_token, v_head;
    const int64_t* positions;
    int64_t pos_stride;
    const int64_t* slots;
    const void* qi;
    int64_t qi_token, qi_head;
    void* qo;
    int64_t qo_token, qo_head;
    uint8_t* k_codes;
    uint8_t* v_codes;
    float* scales;
    int32_t page_rows, n_pages;
    int32_t* err;
};
cudaError_t launch_gqa_append(const GqaAppendCall& c, cudaStream_t stream);

constexpr int kBeamMaxSeq = 65535;   // requests of a selection
size_t beam_workspace_bytes(int32_t n_seq, int32_t n_beams, int64_t vocab, int32_t keep);
cudaError_t launch_beam_select(const void* logits, kvq_dtype dt, int64_t row_stride, int32_t n_seq, int32_t n_beams,
                               int64_t vocab, const float* scores, int32_t keep, float* out_scores, int32_t* parents,
                               int32_t* tokens, void* workspace, cudaStream_t stream);

size_t fork_workspace_bytes(int32_t n_seq, int32_t table_stride, int32_t n_pages);
cudaError_t launch_pages_fork(int32_t n_seq, int32_t page_rows, const int32_t* parents, int64_t* lens, int32_t* table,
                              int32_t table_stride, int32_t* free_pages, int32_t* n_free, int32_t n_pages,
                              int32_t* copies, void* workspace, cudaStream_t stream);
cudaError_t launch_pages_copy(int32_t n, const int32_t* copies, int32_t n_pages, int32_t n_pools,
                              const kvq_pool* pools, int32_t* err, cudaStream_t stream);

}  // namespace kvq
