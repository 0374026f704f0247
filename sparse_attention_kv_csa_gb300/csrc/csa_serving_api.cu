// C entry points of the serving operators (declared in include/csa_serving.h): argument validation, workspace,
// dispatch.
#include "csa_launch.h"
#include "csa_serving_launch.h"

namespace {

using csa::fail_status;

int cuda_status(cudaError_t e, const char *what)
{
    return fail_status(e == cudaErrorMemoryAllocation ? CSA_ERR_OUT_OF_MEMORY : CSA_ERR_CUDA, "%s: %s (%s)", what,
                       cudaGetErrorName(e), cudaGetErrorString(e));
}

int check_ptr(const void *p, const char *name, uintptr_t align)
{
    if (!p)
        return fail_status(CSA_ERR_INVALID_VALUE, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) & (align - 1))
        return fail_status(CSA_ERR_MISALIGNED, "%s = %p is not %d-byte aligned", name, p, (int)align);
    return CSA_OK;
}

int check_opt(const void *p, const char *name, uintptr_t align) { return p ? check_ptr(p, name, align) : CSA_OK; }

int check_stride(int64_t stride, int64_t least, const char *name)
{
    if (stride < least)
        return fail_status(CSA_ERR_INVALID_VALUE, "%s must be at least %lld (got %lld)", name, (long long)least,
                           (long long)stride);
    return CSA_OK;
}

int elem_bytes(int dtype) { return dtype == CSA_DTYPE_F32 ? 4 : dtype == CSA_DTYPE_E4M3 ? 1 : 2; }

#define CSA_TRY(expr)      \
    do {                   \
        int rc_ = (expr);  \
        if (rc_ != CSA_OK) \
            return rc_;    \
    } while (0)

int check_rows(int64_t n_rows, int32_t dim, int32_t dtype)
{
    if (dtype != CSA_DTYPE_BF16 && dtype != CSA_DTYPE_F16 && dtype != CSA_DTYPE_F32)
        return fail_status(CSA_ERR_UNSUPPORTED, "dtype must be bf16, f16 or f32 (got %d)", dtype);
    if (n_rows < 0 || n_rows >= (int64_t(1) << 31))
        return fail_status(CSA_ERR_INVALID_VALUE, "n_rows must be in [0, 2^31) (got %lld)", (long long)n_rows);
    if (dim < 1 || dim > 16384)
        return fail_status(CSA_ERR_UNSUPPORTED, "dim must be in [1, 16384] (got %d)", dim);
    return CSA_OK;
}

// Checks the attentions' common arguments; some: there is something to do, *p filled in.
int check_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride, const int32_t *cu_q,
                    int32_t n_req, int64_t n_tokens, int32_t n_heads, int32_t head_dim, int32_t v_dim,
                    const void *cache, int64_t cache_stride, int32_t cache_dtype, const float *row_scales,
                    int64_t n_pages, int32_t page_size, const int32_t *block_table, int64_t table_stride,
                    int32_t width, const int32_t *seq_lens, int32_t ratio, float scale, const float *sink,
                    void *out, float *lse, csa::AttnParams *p, bool *some)
{
    if (n_req < 0 || n_tokens < 0 || n_heads < 1 || n_pages < 0 || page_size < 1 || width < 0 || ratio < 1)
        return fail_status(CSA_ERR_INVALID_VALUE,
                           "n_req, n_tokens, n_pages and width must be >= 0, n_heads, page_size and ratio >= 1");
    if (head_dim < 8 || head_dim > 1024 || head_dim % 8 != 0 || v_dim < 8 || v_dim > head_dim || v_dim % 8 != 0)
        return fail_status(CSA_ERR_UNSUPPORTED,
                           "head_dim must be a multiple of 8 in [8, 1024] and v_dim one in [8, head_dim] (got %d, %d)",
                           head_dim, v_dim);
    if (cache_dtype != CSA_DTYPE_BF16 && cache_dtype != CSA_DTYPE_E4M3)
        return fail_status(CSA_ERR_UNSUPPORTED, "cache_dtype must be bf16 or e4m3 (got %d)", cache_dtype);
    if (!(scale > 0.0f) || !(scale < 3.0e38f))
        return fail_status(CSA_ERR_INVALID_VALUE, "scale must be positive and finite (got %g)", (double)scale);
    if (n_heads > 4096 || n_tokens >= (int64_t(1) << 31) || n_tokens * (int64_t)n_heads >= (int64_t(1) << 31) || n_req > csa::kMaxRequests)
        return fail_status(CSA_ERR_TOO_LARGE, "n_heads <= 4096, n_tokens * n_heads < 2^31 and n_req <= %d (got %d, %lld, %d)",
                           csa::kMaxRequests, n_heads, (long long)n_tokens, n_req);
    constexpr int64_t kMostRows = (int64_t(1) << 31) - 128;  // (row numbers are rounded up to whole tiles in 32 bits)
    if (n_pages > kMostRows || (int64_t)width * page_size > kMostRows || n_pages * page_size > kMostRows)
        return fail_status(CSA_ERR_TOO_LARGE, "n_pages * page_size and width * page_size must be at most 2^31 - 128");
    CSA_TRY(check_stride(q_head_stride, head_dim, "q_head_stride"));
    CSA_TRY(check_stride(q_token_stride, head_dim, "q_token_stride"));
    CSA_TRY(check_stride(cache_stride, head_dim, "cache_stride"));
    CSA_TRY(check_stride(table_stride, width, "table_stride"));
    if (q_head_stride % 8 || q_token_stride % 8 || cache_stride % (cache_dtype == CSA_DTYPE_E4M3 ? 16 : 8))
        return fail_status(CSA_ERR_MISALIGNED, "the strides of q and cache must be multiples of 16 bytes");
    *some = n_tokens > 0 && n_req > 0;
    if (!*some)
        return CSA_OK;
    CSA_TRY(check_ptr(q, "q", 16));
    CSA_TRY(check_ptr(cu_q, "cu_q", 4));
    CSA_TRY(check_ptr(seq_lens, "seq_lens", 4));
    if (n_pages > 0 && width > 0) {
        CSA_TRY(check_ptr(cache, "cache", 16));
        CSA_TRY(check_ptr(block_table, "block_table", 4));
        if (cache_dtype == CSA_DTYPE_E4M3)
            CSA_TRY(check_ptr(row_scales, "row_scales", 4));
    }
    CSA_TRY(check_opt(sink, "sink", 4));
    CSA_TRY(check_ptr(out, "out", 16));
    CSA_TRY(check_opt(lse, "lse", 4));
    *p = csa::AttnParams{q,       q_token_stride, q_head_stride, cu_q,        n_req,        n_tokens, n_heads, head_dim, v_dim,
                      cache,   cache_stride,   cache_dtype,   cache_dtype == CSA_DTYPE_E4M3 ? row_scales : nullptr,
                      n_pages, page_size,      block_table,   table_stride, n_pages > 0 ? width : 0, seq_lens, ratio, scale, sink,
                      out,     lse,
                      csa::Divider((uint32_t)n_heads), csa::Divider((uint32_t)ratio), csa::Divider((uint32_t)page_size)};
    return CSA_OK;
}

int run_attention(const csa::AttnParams &p, void *stream)
{
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!csa::latent_mma_supported(p)) {
        cudaError_t e = csa::launch_attention_plain(p, st);
        return e == cudaSuccess ? CSA_OK : cuda_status(e, "attention launch");
    }
    int sms = 0;
    cudaMemPool_t pool = nullptr;
    unsigned *status = nullptr;
    cudaError_t e = csa::device_facts(&sms, &pool, &status);
    if (e != cudaSuccess)
        return cuda_status(e, "device set-up");
    void *workspace = nullptr;
    e = cudaMallocFromPoolAsync(&workspace, csa::latent_mma_workspace(p, sms), pool, st);
    if (e != cudaSuccess)
        return cuda_status(e, "attention workspace");
    e = csa::launch_latent_mma(p, workspace, sms, status, st);
    cudaError_t e2 = cudaFreeAsync(workspace, st);
    if (e == cudaSuccess)
        e = e2;
    return e == cudaSuccess ? CSA_OK : cuda_status(e, "attention launch");
}

// Checks the heads that are rotated (none when n_tokens is 0; needed: the table is, for rows) and fills *t in.
int check_turn(const void *x, int64_t x_token_stride, int64_t x_head_stride, const int32_t *positions, int64_t n_tokens,
               int32_t n_heads, int32_t rot_dim, int32_t dtype, const float *rotation, int64_t n_positions, int32_t interleaved,
               int32_t inverse, void *out, int64_t out_token_stride, int64_t out_head_stride, const char *x_name,
               const char *positions_name, bool needed, csa::TurnParams *t)
{
    if (dtype != CSA_DTYPE_BF16 && dtype != CSA_DTYPE_F16 && dtype != CSA_DTYPE_F32)
        return fail_status(CSA_ERR_UNSUPPORTED, "dtype must be bf16, f16 or f32 (got %d)", dtype);
    if (rot_dim < 2 || rot_dim > 1024 || rot_dim % 2 != 0)
        return fail_status(CSA_ERR_UNSUPPORTED, "rot_dim must be even and in [2, 1024] (got %d)", rot_dim);
    if (n_positions < 0 || n_positions > (int64_t(1) << 31) || n_tokens < 0 || (n_tokens > 0 && n_heads < 1))
        return fail_status(CSA_ERR_INVALID_VALUE,
                           "n_positions must be in [0, 2^31], n_tokens >= 0 and n_heads >= 1 (got %lld, %lld, %d)",
                           (long long)n_positions, (long long)n_tokens, n_heads);
    if (n_tokens >= (int64_t(1) << 31) || n_tokens * (int64_t)n_heads >= (int64_t(1) << 31))
        return fail_status(CSA_ERR_TOO_LARGE, "n_tokens * n_heads must be below 2^31 (got %lld, %d)", (long long)n_tokens, n_heads);
    if ((needed || n_tokens > 0) && n_positions > 0)
        CSA_TRY(check_ptr(rotation, "rotation", 4));
    if (n_tokens > 0) {
        const uintptr_t eb = (uintptr_t)elem_bytes(dtype);
        CSA_TRY(check_stride(x_token_stride, rot_dim, "the heads' token stride"));
        CSA_TRY(check_stride(x_head_stride, rot_dim, "the heads' stride"));
        CSA_TRY(check_stride(out_token_stride, rot_dim, "the output's token stride"));
        CSA_TRY(check_stride(out_head_stride, rot_dim, "the output's head stride"));
        CSA_TRY(check_ptr(x, x_name, eb));
        CSA_TRY(check_ptr(positions, positions_name, 4));
        CSA_TRY(check_ptr(out, "the rotated output", eb));
    }
    *t = csa::TurnParams{x,        x_token_stride, x_head_stride, positions, n_tokens, n_tokens > 0 ? n_heads : 1, rot_dim / 2, interleaved != 0,
                         inverse != 0, rotation, n_positions, out, out_token_stride, out_head_stride,
                         csa::Divider((uint32_t)(n_tokens > 0 ? n_heads : 1))};
    return CSA_OK;
}

}  // namespace

extern "C" {

int csa_rms_norm_fwd(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                     const float *weight, int64_t n_rows, int32_t dim, float eps, int32_t dtype, const int64_t *slots,
                     int64_t n_slots, void *out, int64_t out_stride, int32_t out_dtype, float *scales,
                     int32_t scale_group, void *residual_out, float *rstd, void *stream)
{
    CSA_TRY(check_rows(n_rows, dim, dtype));
    if (!(eps >= 0.0f))
        return fail_status(CSA_ERR_INVALID_VALUE, "eps must be >= 0 (got %g)", (double)eps);
    if (out_dtype != dtype && out_dtype != CSA_DTYPE_E4M3)
        return fail_status(CSA_ERR_UNSUPPORTED, "out_dtype must be dtype or e4m3 (got %d)", out_dtype);
    if (scale_group != 0 && (scale_group != 128 || dim % 128 != 0))
        return fail_status(CSA_ERR_UNSUPPORTED, "scale_group must be 0, or 128 with dim a multiple of 128 (got %d, dim %d)",
                           scale_group, dim);
    if (slots && n_slots < 0)
        return fail_status(CSA_ERR_INVALID_VALUE, "n_slots must be >= 0 (got %lld)", (long long)n_slots);
    CSA_TRY(check_stride(x_stride, dim, "x_stride"));
    if (residual)
        CSA_TRY(check_stride(residual_stride, dim, "residual_stride"));
    CSA_TRY(check_stride(out_stride, dim, "out_stride"));
    if (n_rows == 0)
        return CSA_OK;
    const uintptr_t eb = (uintptr_t)elem_bytes(dtype);
    CSA_TRY(check_ptr(x, "x", eb));
    CSA_TRY(check_opt(residual, "residual", eb));
    CSA_TRY(check_opt(weight, "weight", 4));
    CSA_TRY(check_opt(slots, "slots", 8));
    CSA_TRY(check_ptr(out, "out", (uintptr_t)elem_bytes(out_dtype)));
    CSA_TRY(check_opt(residual_out, "residual_out", eb));
    CSA_TRY(check_opt(rstd, "rstd", 4));
    if (out_dtype == CSA_DTYPE_E4M3)
        CSA_TRY(check_ptr(scales, "scales", 4));
    csa::NormFwdParams p{x,     residual,   x_stride,  residual_stride, weight, n_rows, dim, eps, dtype,
                         slots, slots ? n_slots : n_rows, out, out_stride, out_dtype, scales, scale_group,
                         residual_out, rstd, nullptr, 0};
    if (out_dtype == CSA_DTYPE_E4M3 && scale_group == 128 && !csa::norm_fwd_whole_vectors(p))
        return fail_status(CSA_ERR_MISALIGNED, "scale_group 128 needs rows on 16-byte boundaries");
    cudaError_t e = csa::device_facts(nullptr, nullptr, &p.status);
    if (e != cudaSuccess)
        return cuda_status(e, "device set-up");
    e = csa::launch_norm_fwd(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CSA_OK : cuda_status(e, "norm launch");
}

int csa_rms_norm_bwd(const void *h, int64_t h_stride, const void *grad_out, int64_t grad_out_stride,
                     const void *grad_residual, int64_t grad_residual_stride, const float *weight, const float *rstd,
                     int64_t n_rows, int32_t dim, int32_t dtype, void *grad_x, float *grad_weight, void *stream)
{
    CSA_TRY(check_rows(n_rows, dim, dtype));
    CSA_TRY(check_stride(h_stride, dim, "h_stride"));
    CSA_TRY(check_stride(grad_out_stride, dim, "grad_out_stride"));
    if (grad_residual)
        CSA_TRY(check_stride(grad_residual_stride, dim, "grad_residual_stride"));
    CSA_TRY(check_opt(grad_weight, "grad_weight", 4));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (n_rows == 0) {
        if (!grad_weight)
            return CSA_OK;
        cudaError_t e = cudaMemsetAsync(grad_weight, 0, (size_t)dim * sizeof(float), st);
        return e == cudaSuccess ? CSA_OK : cuda_status(e, "grad_weight");
    }
    const uintptr_t eb = (uintptr_t)elem_bytes(dtype);
    CSA_TRY(check_ptr(h, "h", eb));
    CSA_TRY(check_ptr(grad_out, "grad_out", eb));
    CSA_TRY(check_opt(grad_residual, "grad_residual", eb));
    CSA_TRY(check_opt(weight, "weight", 4));
    CSA_TRY(check_ptr(rstd, "rstd", 4));
    CSA_TRY(check_ptr(grad_x, "grad_x", eb));
    csa::NormBwdParams p{h,      grad_out, grad_residual, h_stride, grad_out_stride, grad_residual_stride, weight, rstd,
                         n_rows, dim,      dtype,         grad_x,   grad_weight, nullptr, 0};
    int blocks = 0;
    cudaMemPool_t pool = nullptr;
    cudaError_t e = csa::device_facts(nullptr, &pool, &p.status);
    if (e == cudaSuccess)
        e = csa::norm_bwd_blocks(p, &blocks);
    if (e != cudaSuccess)
        return cuda_status(e, "norm gradient plan");
    void *partial = nullptr;
    e = cudaMallocFromPoolAsync(&partial, (size_t)blocks * dim * sizeof(float), pool, st);
    if (e != cudaSuccess)
        return cuda_status(e, "norm gradient workspace");
    e = csa::launch_norm_bwd(p, static_cast<float *>(partial), st);
    cudaError_t e2 = cudaFreeAsync(partial, st);
    if (e == cudaSuccess)
        e = e2;
    return e == cudaSuccess ? CSA_OK : cuda_status(e, "norm gradient launch");
}

int csa_page_tables(const int32_t *before, const int32_t *after, int32_t n_req, int32_t ratio, int32_t page_size,
                    const int32_t *free_pages, int32_t n_free, const int32_t *taken, const int32_t *table,
                    int64_t table_stride, int32_t width, int64_t capacity, int32_t *table_out, int32_t *cu_rows,
                    int64_t *slots, int32_t *counts, void *stream)
{
    if (n_req < 0 || ratio < 1 || page_size < 1 || n_free < 0 || width < 0 || capacity < 0)
        return fail_status(CSA_ERR_INVALID_VALUE,
                           "n_req, n_free, width and capacity must be >= 0, ratio and page_size >= 1 (got %d, %d, %d, %lld, %d, %d)",
                           n_req, n_free, width, (long long)capacity, ratio, page_size);
    if (n_req > csa::kMaxRequests)
        return fail_status(CSA_ERR_UNSUPPORTED, "n_req must be at most %d (got %d)", csa::kMaxRequests, n_req);
    CSA_TRY(check_stride(table_stride, width, "table_stride"));
    if (n_req > 0) {
        CSA_TRY(check_ptr(before, "before", 4));
        CSA_TRY(check_ptr(after, "after", 4));
        if (width > 0) {
            CSA_TRY(check_ptr(table, "table", 4));
            CSA_TRY(check_ptr(table_out, "table_out", 4));
            if (table == table_out && table_stride != width)
                return fail_status(CSA_ERR_INVALID_VALUE, "table_out may be table only when table_stride == width");
        }
    }
    if (n_free > 0)
        CSA_TRY(check_ptr(free_pages, "free_pages", 4));
    CSA_TRY(check_opt(taken, "taken", 4));
    CSA_TRY(check_ptr(cu_rows, "cu_rows", 4));
    if (capacity > 0)
        CSA_TRY(check_ptr(slots, "slots", 8));
    CSA_TRY(check_ptr(counts, "counts", 4));
    int sms = 0;
    cudaError_t e = csa::device_facts(&sms, nullptr, nullptr);
    if (e != cudaSuccess)
        return cuda_status(e, "device set-up");
    csa::PageParams p{before, after, n_req, ratio, page_size, free_pages, n_free, taken, table, table_stride,
                      width,  capacity, table_out, cu_rows, slots, counts};
    e = csa::launch_page_tables(p, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CSA_OK : cuda_status(e, "page table launch");
}

int csa_latent_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride, const int32_t *cu_q,
                         int32_t n_req, int64_t n_tokens, int32_t n_heads, int32_t head_dim, int32_t v_dim,
                         const void *cache, int64_t cache_stride, int32_t cache_dtype, const float *row_scales,
                         int64_t n_pages, int32_t page_size, const int32_t *block_table, int64_t table_stride,
                         int32_t width, const int32_t *seq_lens, int32_t ratio, float scale, const float *sink,
                         void *out, float *lse, void *stream)
{
    csa::AttnParams p;
    bool some = false;
    CSA_TRY(check_attention(q, q_token_stride, q_head_stride, cu_q, n_req, n_tokens, n_heads, head_dim, v_dim, cache, cache_stride,
                            cache_dtype, row_scales, n_pages, page_size, block_table, table_stride, width, seq_lens, ratio, scale,
                            sink, out, lse, &p, &some));
    return some ? run_attention(p, stream) : CSA_OK;
}

int csa_shared_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride, const int32_t *cu_q,
                         int32_t n_req, int64_t n_tokens, int32_t n_heads, int32_t head_dim, int32_t v_dim,
                         const void *cache, int64_t cache_stride, int32_t cache_dtype, const float *row_scales,
                         int64_t n_pages, int32_t page_size, const int32_t *block_table, int64_t table_stride,
                         int32_t width, const int32_t *seq_lens, const int32_t *cu_groups, const int32_t *shared_rows,
                         int32_t n_groups, int32_t ratio, float scale, const float *sink, void *out, float *lse,
                         void *stream)
{
    if (n_groups < 0)
        return fail_status(CSA_ERR_INVALID_VALUE, "n_groups must be >= 0 (got %d)", n_groups);
    if (n_groups > csa::kMaxRequests)
        return fail_status(CSA_ERR_TOO_LARGE, "n_groups must be at most %d (got %d)", csa::kMaxRequests, n_groups);
    if (n_groups > 0) {
        CSA_TRY(check_ptr(cu_groups, "cu_groups", 4));
        CSA_TRY(check_ptr(shared_rows, "shared_rows", 4));
    }
    csa::AttnParams p;
    bool some = false;
    CSA_TRY(check_attention(q, q_token_stride, q_head_stride, cu_q, n_req, n_tokens, n_heads, head_dim, v_dim, cache, cache_stride,
                            cache_dtype, row_scales, n_pages, page_size, block_table, table_stride, width, seq_lens, ratio, scale,
                            sink, out, lse, &p, &some));
    if (!some)
        return CSA_OK;
    int sms = 0;
    cudaMemPool_t pool = nullptr;
    unsigned *status = nullptr;
    cudaError_t e = csa::device_facts(&sms, &pool, &status);
    if (e != cudaSuccess)
        return cuda_status(e, "device set-up");
    if (!csa::prefix_apart(csa::prefix_call(p, n_groups), sms))
        return run_attention(p, stream);
    e = csa::launch_shared_mma(p, cu_groups, shared_rows, n_groups, sms, pool, status, static_cast<cudaStream_t>(stream));
    if (e == cudaErrorMemoryAllocation) {  // no room for the parts: by request a call needs a few MB, and gives the same
        cudaGetLastError();                // (nor does the next caller of CUDA meet that error)
        return run_attention(p, stream);
    }
    return e == cudaSuccess ? CSA_OK : cuda_status(e, "shared attention launch");
}

int csa_layer_norm_fwd(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride, const float *weight,
                       const float *bias, int64_t n_rows, int32_t dim, float eps, int32_t dtype, void *out, int64_t out_stride,
                       void *residual_out, float *mean, float *rstd, void *stream)
{
    CSA_TRY(check_rows(n_rows, dim, dtype));
    if (!(eps >= 0.0f))
        return fail_status(CSA_ERR_INVALID_VALUE, "eps must be >= 0 (got %g)", (double)eps);
    CSA_TRY(check_stride(x_stride, dim, "x_stride"));
    if (residual)
        CSA_TRY(check_stride(residual_stride, dim, "residual_stride"));
    CSA_TRY(check_stride(out_stride, dim, "out_stride"));
    if (n_rows == 0)
        return CSA_OK;
    const uintptr_t eb = (uintptr_t)elem_bytes(dtype);
    CSA_TRY(check_ptr(x, "x", eb));
    CSA_TRY(check_opt(residual, "residual", eb));
    CSA_TRY(check_opt(weight, "weight", 4));
    CSA_TRY(check_opt(bias, "bias", 4));
    CSA_TRY(check_ptr(out, "out", eb));
    CSA_TRY(check_opt(residual_out, "residual_out", eb));
    CSA_TRY(check_opt(mean, "mean", 4));
    CSA_TRY(check_opt(rstd, "rstd", 4));
    csa::LayerFwdParams p{x,   residual, x_stride, residual_stride, weight, bias, n_rows, dim, eps, dtype,
                          out, out_stride, residual ? residual_out : nullptr, mean, rstd, nullptr, 0};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = csa::device_facts(nullptr, nullptr, &p.status);
    if (e != cudaSuccess)
        return cuda_status(e, "device set-up");
    e = csa::launch_layer_fwd(p, st);
    return e == cudaSuccess ? CSA_OK : cuda_status(e, "layer norm launch");
}

int csa_layer_norm_bwd(const void *h, int64_t h_stride, const void *grad_out, int64_t grad_out_stride, const void *grad_residual,
                       int64_t grad_residual_stride, const float *weight, const float *mean, const float *rstd, int64_t n_rows,
                       int32_t dim, int32_t dtype, void *grad_x, float *grad_weight, float *grad_bias, void *stream)
{
    CSA_TRY(check_rows(n_rows, dim, dtype));
    CSA_TRY(check_stride(h_stride, dim, "h_stride"));
    CSA_TRY(check_stride(grad_out_stride, dim, "grad_out_stride"));
    if (grad_residual)
        CSA_TRY(check_stride(grad_residual_stride, dim, "grad_residual_stride"));
    CSA_TRY(check_opt(grad_weight, "grad_weight", 4));
    CSA_TRY(check_opt(grad_bias, "grad_bias", 4));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (n_rows == 0) {
        cudaError_t e = grad_weight ? cudaMemsetAsync(grad_weight, 0, (size_t)dim * sizeof(float), st) : cudaSuccess;
        if (e == cudaSuccess && grad_bias)
            e = cudaMemsetAsync(grad_bias, 0, (size_t)dim * sizeof(float), st);
        return e == cudaSuccess ? CSA_OK : cuda_status(e, "grad_weight, grad_bias");
    }
    const uintptr_t eb = (uintptr_t)elem_bytes(dtype);
    CSA_TRY(check_ptr(h, "h", eb));
    CSA_TRY(check_ptr(grad_out, "grad_out", eb));
    CSA_TRY(check_opt(grad_residual, "grad_residual", eb));
    CSA_TRY(check_opt(weight, "weight", 4));
    CSA_TRY(check_ptr(mean, "mean", 4));
    CSA_TRY(check_ptr(rstd, "rstd", 4));
    CSA_TRY(check_ptr(grad_x, "grad_x", eb));
    csa::LayerBwdParams p{h, grad_out, grad_residual, h_stride, grad_out_stride, grad_residual_stride, weight, mean, rstd, n_rows,
                          dim, dtype, grad_x, grad_weight, grad_bias, nullptr, 0};
    int blocks = 0;
    cudaMemPool_t pool = nullptr;
    cudaError_t e = csa::device_facts(nullptr, &pool, &p.status);
    if (e == cudaSuccess)
        e = csa::layer_bwd_blocks(p, &blocks);
    if (e != cudaSuccess)
        return cuda_status(e, "layer norm gradient plan");
    void *partial = nullptr;
    e = cudaMallocFromPoolAsync(&partial, (size_t)blocks * 2 * dim * sizeof(float), pool, st);
    if (e != cudaSuccess)
        return cuda_status(e, "layer norm gradient workspace");
    e = csa::launch_layer_bwd(p, static_cast<float *>(partial), st);
    cudaError_t e2 = cudaFreeAsync(partial, st);
    if (e == cudaSuccess)
        e = e2;
    return e == cudaSuccess ? CSA_OK : cuda_status(e, "layer norm gradient launch");
}

int csa_append_rows(const void *rows, int64_t row_stride, int32_t row_dim, const void *rotary, int64_t rotary_stride,
                    int32_t rot_dim, const int32_t *positions, int64_t n_rows, int32_t dtype, const float *rotation,
                    int64_t n_positions, int32_t interleaved, const int64_t *slots, int64_t n_slots, void *out,
                    int64_t out_stride, int32_t out_dtype, float *scales, const void *q, int64_t q_token_stride,
                    int64_t q_head_stride, const int32_t *q_positions, int64_t n_tokens, int32_t n_heads, void *q_out,
                    int64_t q_out_token_stride, int64_t q_out_head_stride, void *stream)
{
    if (n_rows < 0 || n_rows >= (int64_t(1) << 31) || n_slots < 0)
        return fail_status(CSA_ERR_INVALID_VALUE, "n_rows must be in [0, 2^31) and n_slots >= 0 (got %lld, %lld)", (long long)n_rows,
                           (long long)n_slots);
    csa::AppendParams p{};
    CSA_TRY(check_turn(q, q_token_stride, q_head_stride, q_positions, n_tokens, n_heads, rot_dim, dtype, rotation, n_positions,
                       interleaved, false, q_out, q_out_token_stride, q_out_head_stride, "q", "q_positions", n_rows > 0, &p.turn));
    const int64_t width = (int64_t)row_dim + (rotary ? rot_dim : 0);
    if (row_dim < (rotary ? 1 : rot_dim) || width > 1024)
        return fail_status(CSA_ERR_UNSUPPORTED, "row_dim must be at least %d and a row at most 1024 columns (got %d, %lld)",
                           rotary ? 1 : rot_dim, row_dim, (long long)width);
    if (out_dtype != dtype && out_dtype != CSA_DTYPE_E4M3)
        return fail_status(CSA_ERR_UNSUPPORTED, "out_dtype must be dtype or e4m3 (got %d)", out_dtype);
    CSA_TRY(check_stride(row_stride, row_dim, "row_stride"));
    if (rotary)
        CSA_TRY(check_stride(rotary_stride, rot_dim, "rotary_stride"));
    CSA_TRY(check_stride(out_stride, width, "out_stride"));
    const uintptr_t eb = (uintptr_t)elem_bytes(dtype);
    if (n_rows > 0) {
        CSA_TRY(check_ptr(rows, "rows", eb));
        CSA_TRY(check_opt(rotary, "rotary", eb));
        CSA_TRY(check_ptr(positions, "positions", 4));
        CSA_TRY(check_ptr(slots, "slots", 8));
        if (n_slots > 0) {
            CSA_TRY(check_ptr(out, "out", (uintptr_t)elem_bytes(out_dtype)));
            if (out_dtype == CSA_DTYPE_E4M3)
                CSA_TRY(check_ptr(scales, "scales", 4));
        }
    } else if (n_tokens == 0) {
        return CSA_OK;
    }
    p.plain = rows;
    p.plain_stride = row_stride;
    p.plain_dim = rotary ? row_dim : row_dim - rot_dim;
    p.part = rotary ? rotary : static_cast<const uint8_t *>(rows) + (size_t)(row_dim - rot_dim) * eb;
    p.part_stride = rotary ? rotary_stride : row_stride;
    p.positions = positions;
    p.n_rows = n_slots > 0 ? n_rows : 0;
    p.dtype = dtype;
    p.slots = slots;
    p.n_slots = n_slots;
    p.out = out;
    p.out_stride = out_stride;
    p.out_dtype = out_dtype;
    p.scales = scales;
    if (p.n_rows == 0 && n_tokens == 0)
        return CSA_OK;
    cudaError_t e = csa::launch_append(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CSA_OK : cuda_status(e, "append launch");
}

int csa_rotate(const void *x, int64_t x_token_stride, int64_t x_head_stride, const int32_t *positions, int64_t n_tokens,
               int32_t n_heads, int32_t rot_dim, int32_t dtype, const float *rotation, int64_t n_positions, int32_t interleaved,
               int32_t inverse, void *out, int64_t out_token_stride, int64_t out_head_stride, void *stream)
{
    csa::AppendParams p{};
    CSA_TRY(check_turn(x, x_token_stride, x_head_stride, positions, n_tokens, n_heads, rot_dim, dtype, rotation, n_positions,
                       interleaved, inverse, out, out_token_stride, out_head_stride, "x", "positions", false, &p.turn));
    if (n_tokens == 0)
        return CSA_OK;
    p.dtype = p.out_dtype = dtype;
    cudaError_t e = csa::launch_append(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CSA_OK : cuda_status(e, "rotation launch");
}

}  // extern "C"
