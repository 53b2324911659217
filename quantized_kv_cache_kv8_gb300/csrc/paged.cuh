// paged.cuh -- launches of the paged-pool operators, for the C entry points: page
// bookkeeping (pages.cu), rotary append (rope.cu), attention (attn_paged.cu,
// attn_tc_paged.cu).
#pragma once

#include "attn_common.cuh"

#include <utility>

namespace kvq {

// The kernels of a serving step follow one another, each a few microseconds, so each
// is launched while the one before it runs (a launch gap less, about 1.5 us).  Every
// kernel lets its successor come at once and, before it touches global memory, waits
// for its predecessor to have completed, which had waited for its own.  What a
// predecessor may have written it reads by ordinary loads: one through the non-coherent
// path (__ldg) is for what nobody writes while the kernel lives.
template <class K, class... A>
cudaError_t launch_chained(K* kernel, dim3 grid, unsigned block, size_t smem, cudaStream_t stream, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

cudaError_t launch_pages_reserve(int32_t n_seq, int32_t page_rows, const int64_t* lens, const int64_t* new_lens,
                                 int32_t* table, int32_t table_stride, int32_t* free_pages, int32_t* n_free,
                                 int32_t n_pages, int64_t* lens_out, int64_t* cu_new, int64_t* slots,
                                 int64_t* positions, int64_t max_new, void* workspace, cudaStream_t stream);
cudaError_t launch_pages_trim(int32_t n_seq, int32_t page_rows, int64_t* lens, const int64_t* keep, int32_t* table,
                              int32_t table_stride, int32_t* free_pages, int32_t* n_free, int32_t n_pages,
                              void* workspace, cudaStream_t stream);
cudaError_t launch_rope_append(kvq_format fmt, const kvq_mla_layout& L, const kvq_rope& rope, const void* x,
                               kvq_dtype xt, int64_t x_stride, int64_t n, const int64_t* pos, int64_t pos_stride,
                               const int64_t* slots, const void* qi, kvq_dtype qt, int64_t qi_tok, int64_t qi_head,
                               void* qo, int64_t qo_tok, int64_t qo_head, int32_t n_heads, uint8_t* codes,
                               float* scales, int64_t pool_rows, int32_t* err, cudaStream_t stream);
size_t paged_workspace_bytes(bool tensor);
cudaError_t launch_attn_paged(kvq_format fmt, const kvq_mla_layout& L, bool tensor, const void* q, kvq_dtype dt,
                              int64_t n_tok, int32_t n_heads, int32_t n_seq, const int64_t* cu_q, const uint8_t* codes,
                              const float* scales, const int32_t* table, int32_t table_stride,
                              const int64_t* kv_lens, int32_t page_rows, int32_t n_pages, float sm_scale, void* out,
                              void* workspace, cudaStream_t stream);

}  // namespace kvq
