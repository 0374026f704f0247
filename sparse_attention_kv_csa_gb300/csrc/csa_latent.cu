// Attention over a paged cache of shared latent rows, for widths that the tensor-core kernel does not take: a warp a
// (token, head), its query and output in registers, the request's visible rows read one after another.
//
//   s_j = scale q.k_j;  m, l, o updated per row:  m' = max(m, s_j), o = o e^(m-m') + e^(s_j-m') v_j, l likewise
//
// A row's products are summed over the lanes by shuffles, so the time is set by that chain, not by the bytes; four
// rows are taken at a time so that four chains overlap.
#include <cuda_fp8.h>

#include "csa_device.cuh"
#include "csa_launch.h"
#include "csa_serving_launch.h"

namespace csa {
namespace {

constexpr int kWarps = 4;
constexpr int kRows = 4;

__device__ __forceinline__ float2 pair_at(const __nv_bfloat16 *row, int c)
{
    return bf16x2_to_f2(__ldg(reinterpret_cast<const unsigned *>(row + c)));
}

__device__ __forceinline__ float2 pair_at(const __nv_fp8_storage_t *row, int c)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__ldg(reinterpret_cast<const unsigned short *>(row + c)), __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// NP: column pairs a lane holds (columns 64 i + 2 lane)
template <typename C, int NP> __global__ void __launch_bounds__(kWarps * 32) attention_plain_kernel(const AttnParams p)
{
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t token = unit / p.n_heads;
    const int head = (int)(unit % p.n_heads);
    if (token >= p.n_tokens || token >= __ldg(p.cu_q + p.n_req) || token < __ldg(p.cu_q))
        return;
    const int r = find_segment(p.cu_q, p.n_req, (int)token);
    const int end = __ldg(p.cu_q + r + 1);
    const int64_t held = (int64_t)__ldg(p.seq_lens + r) - (end - token) + 1;
    const int64_t most = (int64_t)p.width * p.page_size;
    const int rows = (int)(held < 0 ? 0 : min(held / p.ratio, most));
    float2 q[NP], o[NP];
    const __nv_bfloat16 *qr = static_cast<const __nv_bfloat16 *>(p.q) + token * p.q_token_stride + head * p.q_head_stride;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int c = 64 * i + 2 * lane;
        q[i] = c < p.head_dim ? pair_at(qr, c) : make_float2(0.f, 0.f);
        o[i] = make_float2(0.f, 0.f);
    }
    const int32_t *table = p.block_table + (int64_t)r * p.table_stride;
    const C *cache = static_cast<const C *>(p.cache);
    const float sink = p.sink ? __ldg(p.sink + head) : -INFINITY;
    float m = sink, l = sink > -INFINITY ? 1.0f : 0.0f;
    for (int j0 = 0; j0 < rows; j0 += kRows) {
        float2 k[kRows][NP];
        float s[kRows], f[kRows];
        bool seen[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int j = j0 + u;
            seen[u] = j < rows;
            int64_t slot = 0;
            if (seen[u]) {
                const int page = __ldg(table + j / p.page_size);
                seen[u] = page >= 0 && page < p.n_pages;
                slot = (int64_t)page * p.page_size + j % p.page_size;
            }
            f[u] = 1.0f;
            if (seen[u] && p.row_scales)
                f[u] = __ldg(p.row_scales + slot);
            s[u] = 0.0f;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int c = 64 * i + 2 * lane;
                k[u][i] = seen[u] && c < p.head_dim ? pair_at(cache + slot * p.cache_stride, c) : make_float2(0.f, 0.f);
                s[u] = fmaf(q[i].x, k[u][i].x, s[u]);
                s[u] = fmaf(q[i].y, k[u][i].y, s[u]);
            }
        }
#pragma unroll
        for (int x = 16; x; x >>= 1)
#pragma unroll
            for (int u = 0; u < kRows; ++u)
                s[u] += __shfl_xor_sync(~0u, s[u], x);
        float mn = m;
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            s[u] = seen[u] ? s[u] * f[u] * p.scale : -INFINITY;
            mn = max_nan(mn, s[u]);
        }
        if (mn == -INFINITY)
            continue;  // nothing seen yet
        const float old = expf(m - mn);
        m = mn;
        l *= old;
#pragma unroll
        for (int i = 0; i < NP; ++i)
            o[i] = make_float2(o[i].x * old, o[i].y * old);
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const float e = seen[u] ? expf(s[u] - m) : 0.0f;
            l += e;
            const float ef = e * f[u];
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                o[i].x = fmaf(ef, k[u][i].x, o[i].x);
                o[i].y = fmaf(ef, k[u][i].y, o[i].y);
            }
        }
    }
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + (token * p.n_heads + head) * p.v_dim;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int c = 64 * i + 2 * lane;
        if (c < p.v_dim)
            *reinterpret_cast<unsigned *>(out + c) = f2_to_bf16x2(make_float2(o[i].x * inv, o[i].y * inv));
    }
    if (p.lse && lane == 0)
        p.lse[token * p.n_heads + head] = l > 0.0f || l != l ? m + logf(l) : -INFINITY;
}

template <typename C, int NP> cudaError_t plain_go(const AttnParams &p, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.n_tokens * p.n_heads + kWarps - 1) / kWarps));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attention_plain_kernel<C, NP>, p);
}

template <typename C> cudaError_t plain_size(const AttnParams &p, cudaStream_t st)
{
    if (p.head_dim <= 128) return plain_go<C, 2>(p, st);
    if (p.head_dim <= 256) return plain_go<C, 4>(p, st);
    if (p.head_dim <= 576) return plain_go<C, 9>(p, st);
    return plain_go<C, 16>(p, st);
}

}  // namespace

cudaError_t launch_attention_plain(const AttnParams &p, cudaStream_t st)
{
    return p.cache_dtype == CSA_DTYPE_E4M3 ? plain_size<__nv_fp8_storage_t>(p, st) : plain_size<__nv_bfloat16>(p, st);
}

}  // namespace csa
