// The layer norm's forward (see csa_layer.cuh).  Bound by DRAM where rows are whole vectors: 16411 rows of 4096 with a residual 82.9 us
// in bf16 (96% of the copy rate), 187 in fp32 (85%).  Less with 4-byte loads (4100 columns 149 us, 27%) and narrow rows, of which a warp has one
// (200000 of 128 columns 60 us, 25%).
#include "csa_layer.cuh"

namespace csa {
namespace {

// Every thread of a block runs the same number of rows (idle teams take no row), so the barriers are uniform.
template <typename T, int VEC, int TEAM, int NV, bool STAGED>
__global__ void __launch_bounds__(TEAM < 128 ? 128 : TEAM)
layer_fwd_kernel(const LayerFwdParams p)
{
    constexpr int kThreads = TEAM < 128 ? 128 : TEAM;
    constexpr int kTeams = kThreads / TEAM;
    __shared__ float buf[2][kThreads / 32];
    __shared__ float2 buf2[2][kThreads / 32];
    __shared__ uint64_t all_full[kTeams * kMaxRing];
    extern __shared__ __align__(128) uint8_t ring_mem[];
    const int t = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
    const int arrays = p.residual ? 2 : 1, row_bytes = p.dim * (int)sizeof(T);
    const Ring ring{ring_mem + team * p.stages * arrays * row_bytes, all_full + team * kMaxRing, p.stages, row_bytes, arrays, p.status};
    if (STAGED)
        ring.init(t == 0);
    pdl_wait();
    pdl_trigger();
    const T *x = static_cast<const T *>(p.x), *res = static_cast<const T *>(p.residual);
    float w[NV][VEC], b[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const int c = (i * TEAM + t) * VEC + k;
            w[i][k] = c < p.dim && p.weight ? __ldg(p.weight + c) : 1.0f;
            b[i][k] = c < p.dim && p.bias ? __ldg(p.bias + c) : 0.0f;
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
        if (STAGED || row >= p.n_rows)
            return;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            // short vectors: past the row's end the first one again, as a branch a load would serialise the loads
            int c = (i * TEAM + t) * VEC;
            if (VEC * sizeof(T) < 16)
                c = c < p.dim ? c : 0;
            if (VEC * sizeof(T) < 16 || c < p.dim) {
                nx[i] = load<T, VEC>(x + row * p.x_stride + c);
                if (res)
                    nr[i] = load<T, VEC>(res + row * p.residual_stride + c);
            }
        }
    };
    int64_t row = (int64_t)blockIdx.x * kTeams + team;
    fetch(row);
    if (STAGED && t == 0)
        for (int i = 0; i < ring.stages; ++i)
            refill(row + i * step, i);
    RingAt at;
    for (int64_t it = 0; it < passes; ++it, row += step) {
        const bool live = row < p.n_rows;
        float h[NV][VEC];
        float2 sum = splat(0.0f);
        if (STAGED && live) {
            ring.wait(at, t == 0, row, step, p.n_rows);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TEAM + t) * VEC;
                if (c < p.dim) {
                    nx[i] = from_ring<T, VEC>(ring.at(at.stage, 0), c);
                    if (res)
                        nr[i] = from_ring<T, VEC>(ring.at(at.stage, 1), c);
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
                sum = sum_add(h[i], sum);
            }
        }
        fetch(row + step);
        const float mu = team_reduce<TEAM, false>(sum.x + sum.y, buf[it & 1]) * inv_dim;
        if (STAGED) {
            // the sum's barrier: the whole team has read the stage
            if (TEAM <= 32)
                __syncwarp();
            if (t == 0 && at.ok)
                refill(row + ring.stages * step, at.stage);
            ring.next(at);
        }
        float2 ss = splat(0.0f), rest = splat(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (live && (i * TEAM + t) * VEC < p.dim) {
                add_to(h[i], -mu);
                ss = dot_add(h[i], h[i], ss);
                rest = sum_add(h[i], rest);
            }
        const float2 second = mul2(team_sum2<TEAM>(make_float2(ss.x + ss.y, rest.x + rest.y), buf2[it & 1]), splat(inv_dim));
        const float off = second.y, var = fmaf(-off, off, second.x);
        const float rstd = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + p.eps);  // (NaN stays)
        if (!live)
            continue;
        if (t == 0) {
            if (p.mean)
                p.mean[row] = mu + off;
            if (p.rstd)
                p.rstd[row] = rstd;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TEAM + t) * VEC;
            if (c < p.dim) {
                scale_add(h[i], rstd, -off * rstd);
                fma_by(h[i], w[i], b[i]);
                store<T, VEC>(static_cast<T *>(p.out) + row * p.out_stride + c, pack<T, VEC>(h[i]));
            }
        }
    }
}

template <typename T, int VEC, int TEAM, int NV> cudaError_t fwd_go(LayerFwdParams p, cudaStream_t st)
{
    constexpr int threads = TEAM < 128 ? 128 : TEAM;
    auto k = layer_fwd_kernel<T, VEC, TEAM, NV, false>;
    size_t smem = 0;
    int grid = 0;
    cudaError_t e = norm_plan(k, layer_fwd_kernel<T, VEC, TEAM, NV, VEC * sizeof(T) == 16>, threads, threads / TEAM,
                              p.dim * (int)sizeof(T), p.residual ? 2 : 1, kRingForward, p.n_rows, &k, &p.stages, &smem, &grid);
    return e == cudaSuccess ? launch_pdl(k, dim3(grid), dim3(threads), smem, st, p) : e;
}

template <typename T> cudaError_t fwd_size(const LayerFwdParams &p, int vec, cudaStream_t st)
{
    constexpr int V = 16 / sizeof(T);
    if (vec == V) {
        const int words = p.dim / V;
        if (words <= 32) return fwd_go<T, V, 32, 1>(p, st);
        if (words <= 64) return fwd_go<T, V, 32, 2>(p, st);
        if (words <= 128) return fwd_go<T, V, 64, 2>(p, st);
        if (words <= 256) return fwd_go<T, V, 128, 2>(p, st);
        if (words <= 512) return fwd_go<T, V, 256, 2>(p, st);
        if (words <= 1024) return fwd_go<T, V, 512, 2>(p, st);
        if constexpr (V == 4)  // (16384 columns of 16 bits are 2048 words)
            if (words > 2048) return fwd_go<T, V, 1024, 4>(p, st);
        return fwd_go<T, V, 1024, 2>(p, st);
    }
    if constexpr (sizeof(T) == 2)
        if (vec == 2) {
            if (p.dim <= 512) return fwd_go<T, 2, 64, 4>(p, st);
            if (p.dim <= 2048) return fwd_go<T, 2, 128, 8>(p, st);
            if (p.dim <= 8192) return fwd_go<T, 2, 512, 8>(p, st);
            return fwd_go<T, 2, 1024, 8>(p, st);
        }
    if (p.dim <= 256) return fwd_go<T, 1, 32, 8>(p, st);
    if (p.dim <= 1024) return fwd_go<T, 1, 128, 8>(p, st);
    if (p.dim <= 4096) return fwd_go<T, 1, 512, 8>(p, st);
    return fwd_go<T, 1, 1024, 16>(p, st);
}

}  // namespace

cudaError_t launch_layer_fwd(const LayerFwdParams &p, cudaStream_t st)
{
    const int vec = widest(p.dtype, [&](int v) {
        const int b = v * elem_bytes(p.dtype);
        return p.dim % v == 0 && p.x_stride % v == 0 && on(p.x, b) &&
               (!p.residual || (p.residual_stride % v == 0 && on(p.residual, b))) && on(p.residual_out, b) &&
               p.out_stride % v == 0 && on(p.out, b);
    });
    switch (p.dtype) {
    case CSA_DTYPE_BF16: return fwd_size<__nv_bfloat16>(p, vec, st);
    case CSA_DTYPE_F16: return fwd_size<__half>(p, vec, st);
    default: return fwd_size<float>(p, vec, st);
    }
}

}  // namespace csa
