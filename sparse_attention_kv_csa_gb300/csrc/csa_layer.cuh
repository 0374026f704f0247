// Layer norm with the residual's addition, forward and backward.
//
//   h = round_T(x + r)                      (h = x without a residual)
//   mu = mean_j h_j,  rstd = 1 / sqrt(mean_j (h_j - mu)^2 + eps),  u_j = (h_j - mu) rstd
//   y_j = u_j w_j + b_j,  out = round_T(y)
//
// and from dy and the gradient dh_out that reaches h along the residual stream:
//
//   g_j = w_j dy_j,  dh_j = rstd (g_j - mean(g) - u_j mean(g u)) + dh_out_j;  dx = dr = dh
//   dw_j = sum over rows of dy_j u_j,  db_j = sum over rows of dy_j
//
// The variance is the mean square of the differences from mu, not mean(h^2) - mu^2: the row lies in registers, so the second
// pass over it costs one more reduction and no bytes.  That pass also sums the differences themselves: their mean is what mu's
// rounding left out, which an offset far larger than the spread makes as large as the spread (without it rows of one value came
// out up to 0.9 off zero: 4100 columns of 13891.14 in fp32; 0.29 for 1000 of 10304 in bf16).  Rows, teams, rings, vectors
// and the partial sums of the parameters' gradients are the root-mean-square norm's (csa_norm.cuh).
#pragma once

#include "csa_norm.cuh"

namespace csa {
namespace {

// Both sums over a team of TEAM threads, the same values and order in every thread.  buf: one pair per warp of the block, not
// in use by an earlier unfinished call.
template <int TEAM> __device__ __forceinline__ float2 team_sum2(float2 v, float2 *buf)
{
#pragma unroll
    for (int o = TEAM < 32 ? TEAM / 2 : 16; o; o >>= 1)
        v = add2(v, make_float2(__shfl_xor_sync(~0u, v.x, o), __shfl_xor_sync(~0u, v.y, o)));
    if constexpr (TEAM > 32) {
        constexpr int W = TEAM / 32;
        const int warp = threadIdx.x >> 5, first = warp & ~(W - 1);
        if ((threadIdx.x & 31) == 0)
            buf[warp] = v;
        __syncthreads();
        v = buf[first];
#pragma unroll
        for (int i = 1; i < W; ++i)
            v = add2(v, buf[first + i]);
    }
    return v;
}

template <int VEC> __device__ __forceinline__ void fma_by(float (&v)[VEC], const float (&a)[VEC], const float (&b)[VEC])
{
    if constexpr (VEC > 1) {
#pragma unroll
        for (int k = 0; k < VEC; k += 2) {
            const float2 r = fma2(make_float2(v[k], v[k + 1]), make_float2(a[k], a[k + 1]), make_float2(b[k], b[k + 1]));
            v[k] = r.x;
            v[k + 1] = r.y;
        }
    } else {
        v[0] = fmaf(v[0], a[0], b[0]);
    }
}

template <int VEC> __device__ __forceinline__ void scale_add(float (&v)[VEC], float a, float b)
{
    if constexpr (VEC > 1) {
#pragma unroll
        for (int k = 0; k < VEC; k += 2) {
            const float2 r = fma2(make_float2(v[k], v[k + 1]), splat(a), splat(b));
            v[k] = r.x;
            v[k + 1] = r.y;
        }
    } else {
        v[0] = fmaf(v[0], a, b);
    }
}

template <int VEC> __device__ __forceinline__ void add_to(float (&v)[VEC], float a)
{
    if constexpr (VEC > 1) {
#pragma unroll
        for (int k = 0; k < VEC; k += 2) {
            const float2 r = add2(make_float2(v[k], v[k + 1]), splat(a));
            v[k] = r.x;
            v[k + 1] = r.y;
        }
    } else {
        v[0] += a;
    }
}

template <int VEC> __device__ __forceinline__ float2 sum_add(const float (&a)[VEC], float2 c)
{
    if constexpr (VEC > 1) {
#pragma unroll
        for (int k = 0; k < VEC; k += 2)
            c = add2(make_float2(a[k], a[k + 1]), c);
    } else {
        c.x += a[0];
    }
    return c;
}

}  // namespace
}  // namespace csa
