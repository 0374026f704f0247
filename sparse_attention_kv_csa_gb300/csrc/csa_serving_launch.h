// Launchers of the serving operators (include/csa_serving.h); arguments are validated by the C entry points.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "csa_latent_cuts.h"
#include "csa_serving.h"

namespace csa {

struct NormFwdParams {
    const void *x, *residual;
    int64_t x_stride, residual_stride;
    const float *weight;
    int64_t n_rows;
    int dim;
    float eps;
    int dtype;
    const int64_t *slots;
    int64_t n_slots;  // rows of out
    void *out;
    int64_t out_stride;
    int out_dtype;
    float *scales;
    int scale_group;
    void *residual_out;
    float *rstd;
    unsigned *status;
    int stages;  // (set by the launcher) rows in a block's ring
};
bool norm_fwd_whole_vectors(const NormFwdParams &p);
cudaError_t launch_norm_fwd(const NormFwdParams &p, cudaStream_t st);

struct NormBwdParams {
    const void *h, *grad_out, *grad_residual;
    int64_t h_stride, grad_out_stride, grad_residual_stride;
    const float *weight, *rstd;
    int64_t n_rows;
    int dim, dtype;
    void *grad_x;
    float *grad_weight;
    unsigned *status;
    int stages;  // (set by the launcher) rows in a block's ring
};
// blocks of the launch on the current device = rows of [blocks, dim] partial sums that it writes
cudaError_t norm_bwd_blocks(const NormBwdParams &p, int *blocks);
cudaError_t launch_norm_bwd(const NormBwdParams &p, float *partial, cudaStream_t st);

struct PageParams {
    const int32_t *before, *after;
    int n_req, ratio, page_size;
    const int32_t *free_pages;
    int n_free;
    const int32_t *taken, *table;
    int64_t table_stride;
    int width;
    int64_t capacity;
    int32_t *table_out, *cu_rows;
    int64_t *slots;
    int32_t *counts;
};
constexpr int kMaxRequests = 14000;  // two prefix sums of this length fit an SM's shared memory
cudaError_t launch_page_tables(const PageParams &p, int num_sms, cudaStream_t st);

struct AttnParams {
    const void *q;
    int64_t q_token_stride, q_head_stride;
    const int32_t *cu_q;
    int n_req;
    int64_t n_tokens;
    int n_heads, head_dim, v_dim;
    const void *cache;
    int64_t cache_stride;  // elements
    int cache_dtype;
    const float *row_scales;
    int64_t n_pages;
    int page_size;
    const int32_t *block_table;
    int64_t table_stride;
    int width;
    const int32_t *seq_lens;
    int ratio;
    float scale;
    const float *sink;
    void *out;
    float *lse;
    Divider by_heads, by_ratio, by_page;
};
// Tensor-core kernel: widths in multiples of 64 up to 576 and 512; the workspace holds the parts of split items.
bool latent_mma_supported(const AttnParams &p);
size_t latent_mma_workspace(const AttnParams &p, int num_sms);
cudaError_t launch_latent_mma(const AttnParams &p, void *workspace, int num_sms, unsigned *status, cudaStream_t st);
// Every other width.
cudaError_t launch_attention_plain(const AttnParams &p, cudaStream_t st);

// SM count, workspace pool and status word of the current device (set up on first use).
cudaError_t device_facts(int *num_sms, cudaMemPool_t *pool, unsigned **status);

}  // namespace csa
