// Root-mean-square norm with the residual's addition, forward and backward.
//
//   h = round_T(x + r)                      (h = x without a residual)
//   rstd = 1 / sqrt(mean_j h_j^2 + eps)
//   y_j = h_j rstd w_j
//   out = round_T(y)   or, in 8 bits,  scale_g = max_{j in g} |y_j| / 448,  out = e4m3(y / scale_g)
//
// with g the whole row or 128 columns, and row i stored to row slots[i] of out (a paged cache).  The backward, from
// dy and the gradient dh_out that reaches h along the residual stream:
//
//   c = mean_j(w_j dy_j h_j rstd);  dh_j = rstd (w_j dy_j - h_j rstd c) + dh_out_j;  dx = dr = dh
//   dw_j = sum over rows of dy_j h_j rstd
//
// Both are bound by DRAM: every array is read or written once and a row stays in registers between its sums and its
// output.  A row belongs to one team of 16 to 1024 threads; a block holds one team (or several small ones) and walks
// the rows with the grid's stride, its weights in registers.  Rows of whole 16-byte vectors, where there are more than three
// a resident team, come by bulk copies into a ring of rows in shared memory, several rows ahead (loads into registers a row
// ahead kept too few bytes on the way: 130 against 95 us for 16411 rows of 4096 with 8-bit output); other rows are loaded
// into registers a row ahead.  All sums are fp32; h is rounded to T before the norm because that is what the next layer and
// the backward read.  dw: one partial row per block, added in a fixed order by a second kernel (no atomics).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "csa_device.cuh"
#include "csa_launch.h"
#include "csa_norm_ring.cuh"
#include "csa_serving_launch.h"

namespace csa {
namespace {

constexpr float kE4m3Max = 448.0f;

template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
    static __device__ float to(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __nv_bfloat16 from(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Elem<__half> {
    static __device__ float to(__half v) { return __half2float(v); }
    static __device__ __half from(float v) { return __float2half_rn(v); }
};
template <> struct Elem<float> {
    static __device__ float to(float v) { return v; }
    static __device__ float from(float v) { return v; }
};

// VEC consecutive elements as they lie in memory: 16 bytes, or where widths, strides or bases do not allow that two
// 16-bit elements or one element.
template <typename T, int VEC> struct alignas(VEC == 1 ? sizeof(T) : sizeof(T) * VEC) Pack {
    T v[VEC];
};

// (volatile: the load stays where it is written, ahead of the barriers that it is to overlap)
template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> load(const T *p)
{
    Pack<T, VEC> r;
    if constexpr (VEC * sizeof(T) == 16) {
        uint4 u;
        asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
        memcpy(&r, &u, 16);
    } else if constexpr (VEC * sizeof(T) == 4) {
        uint32_t u;
        asm volatile("ld.global.cs.u32 %0, [%1];" : "=r"(u) : "l"(p));
        memcpy(&r, &u, 4);
    } else {
        static_assert(VEC == 1 && sizeof(T) == 2, "");
        uint16_t u;
        asm volatile("ld.global.cs.u16 %0, [%1];" : "=h"(u) : "l"(p));
        memcpy(&r, &u, 2);
    }
    return r;
}

template <typename T, int VEC> __device__ __forceinline__ void store(T *p, const Pack<T, VEC> &v)
{
    *reinterpret_cast<Pack<T, VEC> *>(p) = v;
}

// A pack's values in fp32 and back (one rounding each), in pairs where the type has them.
template <typename T, int VEC> __device__ __forceinline__ void unpack(const Pack<T, VEC> &a, float (&v)[VEC])
{
    if constexpr (sizeof(T) == 2 && VEC > 1) {
#pragma unroll
        for (int k = 0; k < VEC; k += 2) {
            uint32_t w;
            memcpy(&w, &a.v[k], 4);
            float2 f;
            if constexpr (std::is_same<T, __half>::value)
                f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
            else
                f = bf16x2_to_f2(w);
            v[k] = f.x;
            v[k + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k)
            v[k] = Elem<T>::to(a.v[k]);
    }
}

template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> pack(const float (&v)[VEC])
{
    Pack<T, VEC> a;
    if constexpr (sizeof(T) == 2 && VEC > 1) {
#pragma unroll
        for (int k = 0; k < VEC; k += 2) {
            uint32_t w;
            if constexpr (std::is_same<T, __half>::value) {
                const __half2 h = __floats2half2_rn(v[k], v[k + 1]);
                memcpy(&w, &h, 4);
            } else {
                w = f2_to_bf16x2(make_float2(v[k], v[k + 1]));
            }
            memcpy(&a.v[k], &w, 4);
        }
    } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k)
            a.v[k] = Elem<T>::from(v[k]);
    }
    return a;
}

// Elementwise work in fp32 pairs where there are any: these kernels are bound by instructions as much as by bytes on
// narrow rows (131288 rows of 512 with 8-bit output: 470 instructions a row of a warp without the pairs, 72 us).
template <int VEC> __device__ __forceinline__ void scale_by(float (&v)[VEC], float a)
{
    if constexpr (VEC > 1) {
#pragma unroll
        for (int k = 0; k < VEC; k += 2) {
            const float2 r = mul2(make_float2(v[k], v[k + 1]), splat(a));
            v[k] = r.x;
            v[k + 1] = r.y;
        }
    } else {
        v[0] *= a;
    }
}

template <int VEC> __device__ __forceinline__ void scale_by(float (&v)[VEC], const float (&a)[VEC])
{
    if constexpr (VEC > 1) {
#pragma unroll
        for (int k = 0; k < VEC; k += 2) {
            const float2 r = mul2(make_float2(v[k], v[k + 1]), make_float2(a[k], a[k + 1]));
            v[k] = r.x;
            v[k + 1] = r.y;
        }
    } else {
        v[0] *= a[0];
    }
}

// c + a b, by pairs: c.x takes the even elements, c.y the odd ones.
template <int VEC> __device__ __forceinline__ float2 dot_add(const float (&a)[VEC], const float (&b)[VEC], float2 c)
{
    if constexpr (VEC > 1) {
#pragma unroll
        for (int k = 0; k < VEC; k += 2)
            c = fma2(make_float2(a[k], a[k + 1]), make_float2(b[k], b[k + 1]), c);
    } else {
        c.x = fmaf(a[0], b[0], c.x);
    }
    return c;
}

// Sum (or maximum, NaN if there is one) over a team of TEAM threads, the same value and order in every
// thread.  buf: one float per warp of the block, not in use by an earlier unfinished call.
template <int TEAM, bool MAX> __device__ __forceinline__ float team_reduce(float v, float *buf)
{
#pragma unroll
    for (int o = TEAM < 32 ? TEAM / 2 : 16; o; o >>= 1) {
        const float u = __shfl_xor_sync(~0u, v, o);
        v = MAX ? max_nan(v, u) : v + u;
    }
    if constexpr (TEAM > 32) {
        constexpr int W = TEAM / 32;
        const int warp = threadIdx.x >> 5, first = warp & ~(W - 1);
        if ((threadIdx.x & 31) == 0)
            buf[warp] = v;
        __syncthreads();
        v = buf[first];
#pragma unroll
        for (int i = 1; i < W; ++i)
            v = MAX ? max_nan(v, buf[first + i]) : v + buf[first + i];
    }
    return v;
}

template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> from_ring(const uint8_t *row, int c)
{
    return *reinterpret_cast<const Pack<T, VEC> *>(row + c * sizeof(T));
}

template <typename Kernel, typename... Args>
cudaError_t launch_pdl(Kernel k, dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.dynamicSmemBytes = smem;
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, args...);
}

// Rows in a team's ring: the block's rings 24 KB in the forward (64 KB leave too few blocks an SM: 93 against 79 us for
// 16411 rows of 4096 with 8-bit output) and 40 KB in the backward (28 to 64 KB measured alike), one row where two would
// not fit.  No ring where a team has three rows at most: loads into registers then start sooner (6.5 against 7.6 us for
// 8256 rows of 512 with 8-bit output, some 2.3 rows a team).
constexpr int kRingForward = 24 * 1024, kRingBackward = 40 * 1024;

int ring_stages(int row_bytes, int arrays, int teams, int block_bytes)
{
    const int bytes = row_bytes * arrays * teams, n = block_bytes / bytes;
    return n > kMaxRing ? kMaxRing : n < 2 ? (2 * bytes <= 216 * 1024 ? 2 : 1) : n;
}

// Plans a launch: the ring and a grid of the blocks that are resident at once, or fewer where the rows end sooner.  plain
// and staged are the kernel without and with a ring (the same where vectors are short); *k is the one to launch.
template <typename Kernel>
cudaError_t norm_plan(Kernel plain, Kernel staged, int threads, int teams, int row_bytes, int arrays, int block_bytes,
                      int64_t rows, Kernel *k, int *stages, size_t *smem, int *grid)
{
    const int64_t want = (rows + teams - 1) / teams;
    int resident = 0;
    *k = plain;
    *stages = 0;
    *smem = 0;
    cudaError_t e = resident_blocks(reinterpret_cast<const void *>(plain), threads, 0, 1, &resident);
    if (e == cudaSuccess && plain != staged && want > 3 * (int64_t)resident) {
        *k = staged;
        *stages = ring_stages(row_bytes, arrays, teams, block_bytes);
        *smem = (size_t)*stages * row_bytes * arrays * teams;
        e = resident_blocks(reinterpret_cast<const void *>(staged), threads, *smem, 1, &resident);
    }
    *grid = (int)(want < resident ? want : resident);
    return e;
}

bool on(const void *p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0; }
int elem_bytes(int dtype) { return dtype == CSA_DTYPE_F32 ? 4 : dtype == CSA_DTYPE_E4M3 ? 1 : 2; }

// Elements of a vector: 16 bytes of T where widths, row strides and bases are whole vectors (of the 8-bit output as many
// bytes as elements), else two 16-bit elements, else one.
template <typename Fits> int widest(int dtype, Fits fits)
{
    const int v = 16 / elem_bytes(dtype);
    return fits(v) ? v : elem_bytes(dtype) == 2 && fits(2) ? 2 : 1;
}

}  // namespace
}  // namespace csa
