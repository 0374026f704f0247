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
// output.  A row belongs to one team of 32 to 1024 threads; a block holds one team (or several small ones) and walks
// the rows with the grid's stride, its weights in registers.  Rows of 16-byte vectors for teams of 128 threads or more
// come by bulk copies into a ring of rows in shared memory, several rows ahead (loads into registers a row ahead kept
// too few bytes on the way: 130 against 95 us for 16411 rows of 4096 with 8-bit output); other rows are loaded into
// registers a row ahead.  All sums are fp32; h is rounded to T before the norm because that is what the next layer and
// the backward read.  dw: one partial row per block, added in a fixed order by a second kernel (no atomics).
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "csa_device.cuh"
#include "csa_launch.h"
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

// VEC consecutive elements as they lie in memory (16 bytes, or one element where widths, strides or bases do not
// allow that).
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
    } else {
        static_assert(VEC == 1, "a vector is 16 bytes");
        r.v[0] = *p;
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

// Sum (or NaN-propagating maximum of magnitudes) over a team of TEAM threads, the same value and order in every
// thread.  buf: one float per warp of the block, not in use by an earlier unfinished call.
template <int TEAM, bool MAX> __device__ __forceinline__ float team_reduce(float v, float *buf)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
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

// A ring of rows in shared memory: the arrays' rows side by side, refilled by the block's first thread once the block
// has read them.
struct Ring {
    uint8_t *mem;
    uint64_t *full;
    int stages, row_bytes, arrays;
    unsigned *status;
    __device__ void init() const
    {
        if (threadIdx.x == 0) {
            for (int i = 0; i < stages; ++i)
                mbar_init(smem_addr(full + i), 1);
            mbar_init_fence();
        }
        __syncthreads();
    }
    __device__ void fill(int stage, const void *a, const void *b, const void *c) const
    {
        const uint32_t bar = smem_addr(full + stage), dst = smem_addr(mem) + stage * arrays * row_bytes;
        mbar_arrive_expect_tx(bar, arrays * row_bytes);
        bulk_g2s(dst, a, row_bytes, bar);
        if (b)
            bulk_g2s(dst + row_bytes, b, row_bytes, bar);
        if (c)
            bulk_g2s(dst + (arrays - 1) * row_bytes, c, row_bytes, bar);
    }
    __device__ const uint8_t *at(int stage, int array) const { return mem + (stage * arrays + array) * row_bytes; }
};
constexpr int kMaxRing = 8;

template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> from_ring(const uint8_t *row, int c)
{
    return *reinterpret_cast<const Pack<T, VEC> *>(row + c * sizeof(T));
}

// Every thread of a block runs the same number of rows (idle teams take no row), so the barriers above are uniform.
template <typename T, typename OUT, int VEC, int TEAM, int NV>
__global__ void __launch_bounds__(TEAM < 128 ? 128 : TEAM)
norm_fwd_kernel(const NormFwdParams p)
{
    constexpr int kThreads = TEAM < 128 ? 128 : TEAM;
    constexpr int kTeams = kThreads / TEAM;
    constexpr bool kBits8 = sizeof(OUT) == 1;
    constexpr bool kStaged = VEC > 1 && TEAM >= 128;
    __shared__ float buf[4][kThreads / 32];
    __shared__ uint64_t full[kMaxRing];
    extern __shared__ __align__(128) uint8_t ring_mem[];
    const Ring ring{ring_mem, full, p.stages, p.dim * (int)sizeof(T), p.residual ? 2 : 1, p.status};
    if (kStaged)
        ring.init();
    pdl_wait();
    pdl_trigger();
    const int t = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
    const T *x = static_cast<const T *>(p.x), *res = static_cast<const T *>(p.residual);
    float w[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const int c = (i * TEAM + t) * VEC + k;
            w[i][k] = c < p.dim ? (p.weight ? __ldg(p.weight + c) : 1.0f) : 0.0f;
        }
    const float inv_dim = 1.0f / (float)p.dim;
    const int64_t step = (int64_t)gridDim.x * kTeams;
    const int64_t passes = (p.n_rows + step - 1) / step;
    Pack<T, VEC> nx[NV], nr[NV];
    auto refill = [&](int64_t row, int stage) {
        if (row < p.n_rows)
            ring.fill(stage, x + row * p.x_stride, res ? res + row * p.residual_stride : nullptr, nullptr);
    };
    auto fetch = [&](int64_t row) {
        if (kStaged || row >= p.n_rows)
            return;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TEAM + t) * VEC;
            if (c < p.dim) {
                nx[i] = load<T, VEC>(x + row * p.x_stride + c);
                if (res)
                    nr[i] = load<T, VEC>(res + row * p.residual_stride + c);
            }
        }
    };
    int64_t row = (int64_t)blockIdx.x * kTeams + team;
    fetch(row);
    if (kStaged && threadIdx.x == 0)
        for (int i = 0; i < ring.stages; ++i)
            refill(row + i * step, i);
    int stage = 0;
    uint32_t phase = 0;
    for (int64_t it = 0; it < passes; ++it, row += step) {
        const bool live = row < p.n_rows;
        float h[NV][VEC];
        float ss = 0.0f;
        if (kStaged && live) {
            // (a wait that gives up sets the device's status word; the rows' results are then wrong, as documented)
            mbar_wait(smem_addr(full + stage), phase, ring.status);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TEAM + t) * VEC;
                if (c < p.dim) {
                    nx[i] = from_ring<T, VEC>(ring.at(stage, 0), c);
                    if (res)
                        nr[i] = from_ring<T, VEC>(ring.at(stage, 1), c);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TEAM + t) * VEC;
            if (live && c < p.dim) {
                unpack(nx[i], h[i]);
                if (res) {
                    float r[VEC];
                    unpack(nr[i], r);
#pragma unroll
                    for (int k = 0; k < VEC; ++k)
                        r[k] += h[i][k];
                    const Pack<T, VEC> hp = pack<T, VEC>(r);
                    if (p.residual_out)
                        store<T, VEC>(static_cast<T *>(p.residual_out) + row * p.dim + c, hp);
                    unpack(hp, h[i]);
                }
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    ss = fmaf(h[i][k], h[i][k], ss);
            } else {
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    h[i][k] = 0.0f;
            }
        }
        fetch(row + step);
        ss = team_reduce<TEAM, false>(ss, buf[it & 1]);
        if (kStaged) {
            // the sum's barrier: the whole block has read the stage
            if (threadIdx.x == 0)
                refill(row + ring.stages * step, stage);
            if (++stage == ring.stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        const float rstd = 1.0f / sqrtf(fmaf(ss, inv_dim, p.eps));
        int64_t to = row;
        if (live) {
            if (p.slots)
                to = __ldg(p.slots + row);
            if (p.rstd && t == 0)
                p.rstd[row] = rstd;
        }
        const bool write = live && to >= 0 && to < p.n_slots;
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                h[i][k] = h[i][k] * rstd * w[i][k];
                if (kBits8)
                    amax = max_nan(amax, fabsf(h[i][k]));
            }
        OUT *out = static_cast<OUT *>(p.out) + to * p.out_stride;
        if constexpr (!kBits8) {
            if (write)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = (i * TEAM + t) * VEC;
                    if (c < p.dim)
                        store<OUT, VEC>(out + c, pack<OUT, VEC>(h[i]));
                }
        } else {
            // 128 columns lie in 128 / VEC neighbouring lanes; the host takes that form with whole vectors only
            const bool grouped = VEC > 1 && p.scale_group == 128;
            if (!grouped)
                amax = team_reduce<TEAM, true>(amax, buf[2 + (it & 1)]);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TEAM + t) * VEC;
                if (grouped) {
                    amax = 0.0f;
#pragma unroll
                    for (int k = 0; k < VEC; ++k)
                        amax = max_nan(amax, fabsf(h[i][k]));
#pragma unroll
                    for (int o = 64 / VEC; o; o >>= 1)
                        amax = max_nan(amax, __shfl_xor_sync(~0u, amax, o));
                }
                const float scale = amax / kE4m3Max;
                // y / scale within two roundings of fp32, far below e4m3's half step; a zero row keeps scale 0;
                // a scale whose reciprocal would overflow divides instead
                const bool tiny = scale < 1e-37f;
                const float inv = scale > 0.0f && !tiny ? 1.0f / scale : 1.0f;
                if (write && c < p.dim) {
                    Pack<__nv_fp8_storage_t, VEC> o;
                    if (tiny && scale > 0.0f)
#pragma unroll
                        for (int k = 0; k < VEC; ++k)
                            h[i][k] /= scale;
                    if constexpr (VEC > 1) {
#pragma unroll
                        for (int k = 0; k < VEC; k += 2) {
                            const __nv_fp8x2_storage_t two =
                                __nv_cvt_float2_to_fp8x2(make_float2(h[i][k] * inv, h[i][k + 1] * inv), __NV_SATFINITE, __NV_E4M3);
                            memcpy(&o.v[k], &two, 2);
                        }
                    } else {
                        o.v[0] = __nv_cvt_float_to_fp8(h[i][0] * inv, __NV_SATFINITE, __NV_E4M3);
                    }
                    store<__nv_fp8_storage_t, VEC>(reinterpret_cast<__nv_fp8_storage_t *>(out) + c, o);
                    if (grouped ? (c & 127) == 0 : c == 0)
                        p.scales[to * (grouped ? p.dim / 128 : 1) + (grouped ? c / 128 : 0)] = scale;
                }
            }
        }
    }
}

// Teams of 1024 threads (rows of more than 1024 vectors) have 64 registers a thread: they do not keep the weights.
template <typename T, int VEC, int TEAM, int NV>
__global__ void __launch_bounds__(TEAM < 256 ? 256 : TEAM)
norm_bwd_kernel(const NormBwdParams p, float *__restrict__ partial)
{
    constexpr int kThreads = TEAM < 256 ? 256 : TEAM;
    constexpr int kTeams = kThreads / TEAM;
    constexpr bool kRoomy = TEAM < 1024;
    constexpr bool kStaged = VEC > 1 && TEAM >= 128 && kTeams == 1;
    __shared__ uint64_t full[kMaxRing];
    extern __shared__ __align__(128) uint8_t ring_mem[];
    const Ring ring{ring_mem, full, p.stages, p.dim * (int)sizeof(T), p.grad_residual ? 3 : 2, p.status};
    if (kStaged)
        ring.init();
    __shared__ float buf[2][kThreads / 32];
    __shared__ float fold[kTeams > 1 ? (kTeams - 1) * TEAM * NV * VEC : 1];
    pdl_wait();
    pdl_trigger();
    const int t = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
    const T *h = static_cast<const T *>(p.h), *dy = static_cast<const T *>(p.grad_out);
    const T *dh = static_cast<const T *>(p.grad_residual);
    auto weight_at = [&](int i, int k) {
        const int c = (i * TEAM + t) * VEC + k;
        return c < p.dim ? (p.weight ? __ldg(p.weight + c) : 1.0f) : 0.0f;
    };
    float w[NV][VEC], dw[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            if (kRoomy)
                w[i][k] = weight_at(i, k);
            dw[i][k] = 0.0f;
        }
    const float inv_dim = 1.0f / (float)p.dim;
    const int64_t step = (int64_t)gridDim.x * kTeams;
    const int64_t passes = (p.n_rows + step - 1) / step;
    int64_t row = (int64_t)blockIdx.x * kTeams + team;
    struct Row {
        Pack<T, VEC> h[NV], g[NV], r[NV];
        float rstd;
    };
    auto fetch = [&](int64_t r, Row &x) {
        if (r >= p.n_rows)
            return;
        x.rstd = __ldg(p.rstd + r);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TEAM + t) * VEC;
            if (c < p.dim) {
                x.h[i] = load<T, VEC>(h + r * p.h_stride + c);
                x.g[i] = load<T, VEC>(dy + r * p.grad_out_stride + c);
                if (dh)
                    x.r[i] = load<T, VEC>(dh + r * p.grad_residual_stride + c);
            }
        }
    };
    // unit = h rstd, g = w dy
    auto values = [&](const Row &x, int i, float (&unit)[VEC], float (&g)[VEC], float (&raw)[VEC]) {
        unpack(x.h[i], unit);
        unpack(x.g[i], raw);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            unit[k] *= x.rstd;
            g[k] = raw[k] * (kRoomy ? w[i][k] : weight_at(i, k));
        }
    };
    Row now, next;
    auto refill = [&](int64_t r, int stage) {
        if (r < p.n_rows)
            ring.fill(stage, h + r * p.h_stride, dy + r * p.grad_out_stride, dh ? dh + r * p.grad_residual_stride : nullptr);
    };
    if (kStaged) {
        if (threadIdx.x == 0)
            for (int i = 0; i < ring.stages; ++i)
                refill(row + i * step, i);
    } else if (kRoomy) {
        fetch(row, next);
    }
    int stage = 0;
    uint32_t phase = 0;
    for (int64_t it = 0; it < passes; ++it, row += step) {
        const bool live = row < p.n_rows;
        if (kStaged) {
            if (live) {
                now.rstd = __ldg(p.rstd + row);
                mbar_wait(smem_addr(full + stage), phase, ring.status);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = (i * TEAM + t) * VEC;
                    if (c < p.dim) {
                        now.h[i] = from_ring<T, VEC>(ring.at(stage, 0), c);
                        now.g[i] = from_ring<T, VEC>(ring.at(stage, 1), c);
                        if (dh)
                            now.r[i] = from_ring<T, VEC>(ring.at(stage, 2), c);
                    }
                }
            }
        } else if (kRoomy) {
            now = next;
            fetch(row + step, next);
        } else {
            fetch(row, now);
        }
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (live && (i * TEAM + t) * VEC < p.dim) {
                float unit[VEC], g[VEC], raw[VEC];
                values(now, i, unit, g, raw);
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    dw[i][k] = fmaf(raw[k], unit[k], dw[i][k]);
                    sum = fmaf(g[k], unit[k], sum);
                }
            }
        const float c_mean = team_reduce<TEAM, false>(sum, buf[it & 1]) * inv_dim;
        if (kStaged) {
            if (threadIdx.x == 0)
                refill(row + ring.stages * step, stage);
            if (++stage == ring.stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TEAM + t) * VEC;
            if (live && c < p.dim) {
                float unit[VEC], g[VEC], raw[VEC], d[VEC];
                values(now, i, unit, g, raw);
                if (dh)
                    unpack(now.r[i], raw);
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    d[k] = now.rstd * fmaf(-unit[k], c_mean, g[k]);
                    if (dh)
                        d[k] += raw[k];
                }
                store<T, VEC>(static_cast<T *>(p.grad_x) + row * p.dim + c, pack<T, VEC>(d));
            }
        }
    }
    if constexpr (kTeams > 1) {
        // the teams' sums of one block, added in ascending team order
        if (team > 0)
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    fold[((team - 1) * NV * VEC + i * VEC + k) * TEAM + t] = dw[i][k];
        __syncthreads();
        if (team == 0)
            for (int u = 0; u < kTeams - 1; ++u)
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int k = 0; k < VEC; ++k)
                        dw[i][k] += fold[(u * NV * VEC + i * VEC + k) * TEAM + t];
    }
    if (team == 0)
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const int c = (i * TEAM + t) * VEC + k;
                if (c < p.dim)
                    partial[(int64_t)blockIdx.x * p.dim + c] = dw[i][k];
            }
}

// dw[c] = the partial rows' sum: 32 lanes of rows a column, each in ascending order, then the lanes in order.
__global__ void __launch_bounds__(1024) norm_dweight_kernel(const float *__restrict__ partial, int n_partials, int dim,
                                                            float *__restrict__ dweight)
{
    __shared__ float sums[32][33];
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.0f;
    if (c < dim)
        for (int r = threadIdx.y; r < n_partials; r += 32)
            s += partial[(int64_t)r * dim + c];
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    float v = sums[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(~0u, v, o);
    const int cw = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && cw < dim)
        dweight[cw] = v;
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

// Persistent grid: as many blocks as are resident at once, or fewer where the rows end sooner.
template <typename Kernel> cudaError_t norm_grid(Kernel k, int threads, int teams, size_t smem, int64_t rows, int *grid)
{
    int resident = 0;
    cudaError_t e = resident_blocks(reinterpret_cast<const void *>(k), threads, smem, 1, &resident);
    const int64_t want = (rows + teams - 1) / teams;
    *grid = (int)(want < resident ? want : resident);
    return e;
}

// Rows in a block's ring: about 64 KB, so that three or four blocks' rings fill an SM's shared memory; one row where
// two would not fit.
int ring_stages(int row_bytes, int arrays, int64_t rows)
{
    const int bytes = row_bytes * arrays;
    int n = (64 * 1024) / bytes;
    n = n > kMaxRing ? kMaxRing : n < 2 && 2 * bytes <= 216 * 1024 ? 2 : n < 1 ? 1 : n;
    return n > rows ? (int)rows : n;
}

template <typename T, typename OUT, int VEC, int TEAM, int NV>
cudaError_t fwd_go(NormFwdParams p, cudaStream_t st)
{
    constexpr int threads = TEAM < 128 ? 128 : TEAM;
    const int arrays = p.residual ? 2 : 1, row_bytes = p.dim * (int)sizeof(T);
    p.stages = VEC > 1 && TEAM >= 128 ? ring_stages(row_bytes, arrays, p.n_rows) : 0;
    const size_t smem = (size_t)p.stages * arrays * row_bytes;
    int grid = 0;
    cudaError_t e = norm_grid(norm_fwd_kernel<T, OUT, VEC, TEAM, NV>, threads, threads / TEAM, smem, p.n_rows, &grid);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(norm_fwd_kernel<T, OUT, VEC, TEAM, NV>, dim3(grid), dim3(threads), smem, st, p);
}

// A row of `words` vectors (or elements) goes to the smallest team whose threads hold at most four vectors (sixteen
// elements) each: the more a thread holds, the more loads it has in flight and the fewer warps a sum crosses.
template <typename T, typename OUT> cudaError_t fwd_size(const NormFwdParams &p, bool vec, cudaStream_t st)
{
    constexpr int V = 16 / sizeof(T);
    if (vec) {
        const int words = p.dim / V;
        if (words <= 32) return fwd_go<T, OUT, V, 32, 1>(p, st);
        if (words <= 64) return fwd_go<T, OUT, V, 32, 2>(p, st);
        if (words <= 128) return fwd_go<T, OUT, V, 32, 4>(p, st);
        if (words <= 512) return fwd_go<T, OUT, V, 128, 4>(p, st);
        if (words <= 1024) return fwd_go<T, OUT, V, 256, 4>(p, st);
        if (words <= 2048) return fwd_go<T, OUT, V, 512, 4>(p, st);
        return fwd_go<T, OUT, V, 1024, 4>(p, st);
    }
    if (p.dim <= 512) return fwd_go<T, OUT, 1, 32, 16>(p, st);
    if (p.dim <= 2048) return fwd_go<T, OUT, 1, 128, 16>(p, st);
    if (p.dim <= 4096) return fwd_go<T, OUT, 1, 256, 16>(p, st);
    return fwd_go<T, OUT, 1, 1024, 16>(p, st);
}

template <typename T, int VEC, int TEAM, int NV>
cudaError_t bwd_go(NormBwdParams p, float *partial, int *blocks, bool plan, cudaStream_t st)
{
    constexpr int threads = TEAM < 256 ? 256 : TEAM;
    const int arrays = p.grad_residual ? 3 : 2, row_bytes = p.dim * (int)sizeof(T);
    p.stages = VEC > 1 && threads == TEAM ? ring_stages(row_bytes, arrays, p.n_rows) : 0;
    const size_t smem = (size_t)p.stages * arrays * row_bytes;
    int grid = 0;
    cudaError_t e = norm_grid(norm_bwd_kernel<T, VEC, TEAM, NV>, threads, threads / TEAM, smem, p.n_rows, &grid);
    if (e != cudaSuccess)
        return e;
    *blocks = grid;
    return plan ? cudaSuccess : launch_pdl(norm_bwd_kernel<T, VEC, TEAM, NV>, dim3(grid), dim3(threads), smem, st, p, partial);
}

template <typename T>
cudaError_t bwd_size(const NormBwdParams &p, bool vec, float *partial, int *blocks, bool plan, cudaStream_t st)
{
    constexpr int V = 16 / sizeof(T);
    if (vec) {
        const int words = p.dim / V;
        if (words <= 32) return bwd_go<T, V, 32, 1>(p, partial, blocks, plan, st);
        if (words <= 64) return bwd_go<T, V, 32, 2>(p, partial, blocks, plan, st);
        if (words <= 128) return bwd_go<T, V, 64, 2>(p, partial, blocks, plan, st);
        if (words <= 256) return bwd_go<T, V, 128, 2>(p, partial, blocks, plan, st);
        if (words <= 512) return bwd_go<T, V, 256, 2>(p, partial, blocks, plan, st);
        if (words <= 1024) return bwd_go<T, V, 512, 2>(p, partial, blocks, plan, st);
        if (words <= 2048) return bwd_go<T, V, 1024, 2>(p, partial, blocks, plan, st);
        return bwd_go<T, V, 1024, 4>(p, partial, blocks, plan, st);
    }
    if (p.dim <= 256) return bwd_go<T, 1, 32, 8>(p, partial, blocks, plan, st);
    if (p.dim <= 2048) return bwd_go<T, 1, 256, 8>(p, partial, blocks, plan, st);
    if (p.dim <= 8192) return bwd_go<T, 1, 1024, 8>(p, partial, blocks, plan, st);
    return bwd_go<T, 1, 1024, 16>(p, partial, blocks, plan, st);
}

bool on16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
int elem_bytes(int dtype) { return dtype == CSA_DTYPE_F32 ? 4 : dtype == CSA_DTYPE_E4M3 ? 1 : 2; }

}  // namespace

// Whole 16-byte vectors: bases, row strides and the width in 16 bytes of T (the 8-bit output's vectors are 16 / sizeof(T)
// bytes).
bool norm_fwd_vectors(const NormFwdParams &p)
{
    const int v = 16 / elem_bytes(p.dtype);
    const uintptr_t ob = (uintptr_t)v * elem_bytes(p.out_dtype);
    return p.dim % v == 0 && p.x_stride % v == 0 && on16(p.x) &&
           (!p.residual || (p.residual_stride % v == 0 && on16(p.residual))) && on16(p.residual_out) &&
           p.out_stride % v == 0 && reinterpret_cast<uintptr_t>(p.out) % ob == 0;
}

static bool norm_bwd_vectors(const NormBwdParams &p)
{
    const int v = 16 / elem_bytes(p.dtype);
    return p.dim % v == 0 && p.h_stride % v == 0 && on16(p.h) && p.grad_out_stride % v == 0 && on16(p.grad_out) &&
           (!p.grad_residual || (p.grad_residual_stride % v == 0 && on16(p.grad_residual))) && on16(p.grad_x);
}

cudaError_t launch_norm_fwd(const NormFwdParams &p, cudaStream_t st)
{
    const bool vec = norm_fwd_vectors(p), bits8 = p.out_dtype == CSA_DTYPE_E4M3;
    switch (p.dtype) {
    case CSA_DTYPE_BF16:
        return bits8 ? fwd_size<__nv_bfloat16, __nv_fp8_e4m3>(p, vec, st) : fwd_size<__nv_bfloat16, __nv_bfloat16>(p, vec, st);
    case CSA_DTYPE_F16:
        return bits8 ? fwd_size<__half, __nv_fp8_e4m3>(p, vec, st) : fwd_size<__half, __half>(p, vec, st);
    default:
        return bits8 ? fwd_size<float, __nv_fp8_e4m3>(p, vec, st) : fwd_size<float, float>(p, vec, st);
    }
}

static cudaError_t norm_bwd_call(const NormBwdParams &p, float *partial, int *blocks, bool plan, cudaStream_t st)
{
    const bool vec = norm_bwd_vectors(p);
    switch (p.dtype) {
    case CSA_DTYPE_BF16: return bwd_size<__nv_bfloat16>(p, vec, partial, blocks, plan, st);
    case CSA_DTYPE_F16: return bwd_size<__half>(p, vec, partial, blocks, plan, st);
    default: return bwd_size<float>(p, vec, partial, blocks, plan, st);
    }
}

cudaError_t norm_bwd_blocks(const NormBwdParams &p, int *blocks) { return norm_bwd_call(p, nullptr, blocks, true, nullptr); }

cudaError_t launch_norm_bwd(const NormBwdParams &p, float *partial, cudaStream_t st)
{
    int blocks = 0;
    cudaError_t e = norm_bwd_call(p, partial, &blocks, false, st);
    if (e != cudaSuccess || !p.grad_weight)
        return e;
    return launch_pdl(norm_dweight_kernel, dim3((p.dim + 31) / 32), dim3(32, 32), 0, st, partial, blocks, p.dim, p.grad_weight);
}

}  // namespace csa
