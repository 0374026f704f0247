// The layer norm's backward (see csa_layer.cuh).  Bound by DRAM where rows are whole vectors: 16384 rows of 4096 with a residual 97 us in
// bf16 (81% of the copy rate), 176 in fp32 (90%); by short loads and their instructions where they are not (5003 rows of 1001 17.5 us in
// fp16, floor 4.4, and 17.0 in fp32, floor 8.9).
#include "csa_layer.cuh"

namespace csa {
namespace {

// A block's sums for the parameters' gradients go to partial[block]: dim of the weight's, then dim of the bias's.
// Teams of 1024 threads (rows of more than 1024 vectors) have 64 registers a thread: they do not keep the weights.
template <typename T, int VEC, int TEAM, int NV, bool STAGED>
__global__ void __launch_bounds__(TEAM < 256 ? 256 : TEAM)
layer_bwd_kernel(const LayerBwdParams p, float *__restrict__ partial)
{
    constexpr int kThreads = TEAM < 256 ? 256 : TEAM;
    constexpr int kTeams = kThreads / TEAM;
    constexpr bool kRoomy = TEAM < 1024;
    __shared__ uint64_t all_full[kTeams * kMaxRing];
    extern __shared__ __align__(128) uint8_t ring_mem[];
    const int t = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
    const int arrays = p.grad_residual ? 3 : 2, row_bytes = p.dim * (int)sizeof(T);
    const Ring ring{ring_mem + team * p.stages * arrays * row_bytes, all_full + team * kMaxRing, p.stages, row_bytes, arrays, p.status};
    if (STAGED)
        ring.init(t == 0);
    __shared__ float2 buf[2][kThreads / 32];
    __shared__ float fold[kTeams > 1 ? (kTeams - 1) * TEAM * NV * VEC : 1];
    pdl_wait();
    pdl_trigger();
    const T *h = static_cast<const T *>(p.h), *dy = static_cast<const T *>(p.grad_out);
    const T *dh = static_cast<const T *>(p.grad_residual);
    auto weight_at = [&](int i, int k) {
        const int c = (i * TEAM + t) * VEC + k;
        return c < p.dim && p.weight ? __ldg(p.weight + c) : 1.0f;
    };
    float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            if (kRoomy)
                w[i][k] = weight_at(i, k);
            dw[i][k] = db[i][k] = 0.0f;
        }
    const float inv_dim = 1.0f / (float)p.dim;
    const int64_t step = (int64_t)gridDim.x * kTeams;
    const int64_t passes = (p.n_rows + step - 1) / step;
    int64_t row = (int64_t)blockIdx.x * kTeams + team;
    struct Row {
        Pack<T, VEC> h[NV], g[NV], r[NV];
        float rstd, shift;  // shift: -mean (u = (h - mean) rstd; h rstd - mean rstd would lose an offset's digits)
    };
    auto fetch = [&](int64_t r, Row &x) {
        if (r >= p.n_rows)
            return;
        x.rstd = __ldg(p.rstd + r);
        x.shift = -__ldg(p.mean + r);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            // short vectors: past the row's end the first one again, as a branch a load would serialise the loads
            int c = (i * TEAM + t) * VEC;
            if (VEC * sizeof(T) < 16)
                c = c < p.dim ? c : 0;
            if (VEC * sizeof(T) < 16 || c < p.dim) {
                x.h[i] = load<T, VEC>(h + r * p.h_stride + c);
                x.g[i] = load<T, VEC>(dy + r * p.grad_out_stride + c);
                if (dh)
                    x.r[i] = load<T, VEC>(dh + r * p.grad_residual_stride + c);
            }
        }
    };
    // unit = (h - mean) rstd, g = w dy
    auto values = [&](const Row &x, int i, float (&unit)[VEC], float (&g)[VEC], float (&raw)[VEC]) {
        unpack(x.h[i], unit);
        unpack(x.g[i], raw);
        add_to(unit, x.shift);
        scale_by(unit, x.rstd);
#pragma unroll
        for (int k = 0; k < VEC; ++k)
            g[k] = kRoomy ? w[i][k] : weight_at(i, k);
        scale_by(g, raw);
    };
    Row now, next;
    auto refill = [&](int64_t r, int stage) {
        if (r < p.n_rows)
            ring.fill(stage, h + r * p.h_stride, dy + r * p.grad_out_stride, dh ? dh + r * p.grad_residual_stride : nullptr);
    };
    if (STAGED) {
        if (t == 0)
            for (int i = 0; i < ring.stages; ++i)
                refill(row + i * step, i);
    } else if (kRoomy) {
        fetch(row, next);
    }
    RingAt at;
    for (int64_t it = 0; it < passes; ++it, row += step) {
        const bool live = row < p.n_rows;
        if (STAGED) {
            if (live) {
                now.rstd = __ldg(p.rstd + row);
                now.shift = -__ldg(p.mean + row);
                ring.wait(at, t == 0, row, step, p.n_rows);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = (i * TEAM + t) * VEC;
                    if (c < p.dim) {
                        now.h[i] = from_ring<T, VEC>(ring.at(at.stage, 0), c);
                        now.g[i] = from_ring<T, VEC>(ring.at(at.stage, 1), c);
                        if (dh)
                            now.r[i] = from_ring<T, VEC>(ring.at(at.stage, 2), c);
                    }
                }
            }
        } else if (kRoomy) {
            now = next;
            fetch(row + step, next);
        } else {
            fetch(row, now);
        }
        float2 through = splat(0.0f), level = splat(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (live && (i * TEAM + t) * VEC < p.dim) {
                float unit[VEC], g[VEC], raw[VEC];
                values(now, i, unit, g, raw);
                through = dot_add(g, unit, through);
                level = sum_add(g, level);
                fma_by(unit, raw, dw[i]);
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    dw[i][k] = unit[k];
                if constexpr (VEC > 1) {
#pragma unroll
                    for (int k = 0; k < VEC; k += 2) {
                        const float2 s = add2(make_float2(db[i][k], db[i][k + 1]), make_float2(raw[k], raw[k + 1]));
                        db[i][k] = s.x;
                        db[i][k + 1] = s.y;
                    }
                } else {
                    db[i][0] += raw[0];
                }
            }
        float2 mean = team_sum2<TEAM>(make_float2(through.x + through.y, level.x + level.y), buf[it & 1]);
        mean = mul2(mean, splat(inv_dim));
        if (STAGED) {
            if (TEAM == 32)
                __syncwarp();
            if (t == 0 && at.ok)
                refill(row + ring.stages * step, at.stage);
            ring.next(at);
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
                    d[k] = now.rstd * (fmaf(-unit[k], mean.x, g[k]) - mean.y);
                    if (dh)
                        d[k] += raw[k];
                }
                store<T, VEC>(static_cast<T *>(p.grad_x) + row * p.dim + c, pack<T, VEC>(d));
            }
        }
    }
    // the teams' sums of one block, added in ascending team order: the weight's, then the bias's through the same space
    float *mine = partial + (int64_t)blockIdx.x * 2 * p.dim;
    auto put = [&](float (&sum)[NV][VEC], float *dst) {
        if constexpr (kTeams > 1) {
            __syncthreads();
            if (team > 0)
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int k = 0; k < VEC; ++k)
                        fold[((team - 1) * NV * VEC + i * VEC + k) * TEAM + t] = sum[i][k];
            __syncthreads();
            if (team == 0)
                for (int u = 0; u < kTeams - 1; ++u)
#pragma unroll
                    for (int i = 0; i < NV; ++i)
#pragma unroll
                        for (int k = 0; k < VEC; ++k)
                            sum[i][k] += fold[(u * NV * VEC + i * VEC + k) * TEAM + t];
        }
        if (team == 0)
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    const int c = (i * TEAM + t) * VEC + k;
                    if (c < p.dim)
                        dst[c] = sum[i][k];
                }
    };
    put(dw, mine);
    put(db, mine + p.dim);
}

// The partial rows' sums: 32 lanes of rows a column, each in ascending order, then the lanes in order.
__global__ void __launch_bounds__(1024) layer_params_kernel(const float *__restrict__ partial, int n_partials, int dim,
                                                            float *__restrict__ dweight, float *__restrict__ dbias)
{
    __shared__ float sums[32][33];
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.0f;
    if (c < 2 * dim)
        for (int r = threadIdx.y; r < n_partials; r += 32)
            s += partial[(int64_t)r * 2 * dim + c];
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    float v = sums[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(~0u, v, o);
    const int to = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && to < 2 * dim) {
        float *dst = to < dim ? dweight : dbias;
        if (dst)
            dst[to < dim ? to : to - dim] = v;
    }
}

template <typename T, int VEC, int TEAM, int NV>
cudaError_t bwd_go(LayerBwdParams p, float *partial, int *blocks, bool plan, cudaStream_t st)
{
    constexpr int threads = TEAM < 256 ? 256 : TEAM;
    auto k = layer_bwd_kernel<T, VEC, TEAM, NV, false>;
    size_t smem = 0;
    cudaError_t e = norm_plan(k, layer_bwd_kernel<T, VEC, TEAM, NV, VEC * sizeof(T) == 16>, threads, threads / TEAM,
                              p.dim * (int)sizeof(T), p.grad_residual ? 3 : 2, kRingBackward, p.n_rows, &k, &p.stages, &smem,
                              blocks);
    return e != cudaSuccess || plan ? e : launch_pdl(k, dim3(*blocks), dim3(threads), smem, st, p, partial);
}

template <typename T>
cudaError_t bwd_size(const LayerBwdParams &p, int vec, float *partial, int *blocks, bool plan, cudaStream_t st)
{
    constexpr int V = 16 / sizeof(T);
    if (vec == V) {
        const int words = p.dim / V;
        if (words <= 32) return bwd_go<T, V, 32, 1>(p, partial, blocks, plan, st);
        if (words <= 64) return bwd_go<T, V, 32, 2>(p, partial, blocks, plan, st);
        if (words <= 128) return bwd_go<T, V, 64, 2>(p, partial, blocks, plan, st);
        if (words <= 256) return bwd_go<T, V, 128, 2>(p, partial, blocks, plan, st);
        if (words <= 512) return bwd_go<T, V, 256, 2>(p, partial, blocks, plan, st);
        if (words <= 1024) return bwd_go<T, V, 512, 2>(p, partial, blocks, plan, st);
        if constexpr (V == 4)  // (16384 columns of 16 bits are 2048 words)
            if (words > 2048) return bwd_go<T, V, 1024, 4>(p, partial, blocks, plan, st);
        return bwd_go<T, V, 1024, 2>(p, partial, blocks, plan, st);
    }
    if constexpr (sizeof(T) == 2)
        if (vec == 2) {
            if (p.dim <= 512) return bwd_go<T, 2, 64, 4>(p, partial, blocks, plan, st);
            if (p.dim <= 2048) return bwd_go<T, 2, 256, 4>(p, partial, blocks, plan, st);
            if (p.dim <= 4096) return bwd_go<T, 2, 512, 4>(p, partial, blocks, plan, st);
            if (p.dim <= 8192) return bwd_go<T, 2, 512, 8>(p, partial, blocks, plan, st);
            return bwd_go<T, 2, 1024, 8>(p, partial, blocks, plan, st);
        }
    if (p.dim <= 256) return bwd_go<T, 1, 32, 8>(p, partial, blocks, plan, st);
    if (p.dim <= 1024) return bwd_go<T, 1, 128, 8>(p, partial, blocks, plan, st);
    if (p.dim <= 4096) return bwd_go<T, 1, 512, 8>(p, partial, blocks, plan, st);
    return bwd_go<T, 1, 1024, 16>(p, partial, blocks, plan, st);
}

cudaError_t bwd_call(const LayerBwdParams &p, float *partial, int *blocks, bool plan, cudaStream_t st)
{
    const int vec = widest(p.dtype, [&](int v) {
        const int b = v * elem_bytes(p.dtype);
        return p.dim % v == 0 && p.h_stride % v == 0 && on(p.h, b) && p.grad_out_stride % v == 0 && on(p.grad_out, b) &&
               (!p.grad_residual || (p.grad_residual_stride % v == 0 && on(p.grad_residual, b))) && on(p.grad_x, b);
    });
    switch (p.dtype) {
    case CSA_DTYPE_BF16: return bwd_size<__nv_bfloat16>(p, vec, partial, blocks, plan, st);
    case CSA_DTYPE_F16: return bwd_size<__half>(p, vec, partial, blocks, plan, st);
    default: return bwd_size<float>(p, vec, partial, blocks, plan, st);
    }
}

}  // namespace

cudaError_t layer_bwd_blocks(const LayerBwdParams &p, int *blocks) { return bwd_call(p, nullptr, blocks, true, nullptr); }

cudaError_t launch_layer_bwd(const LayerBwdParams &p, float *partial, cudaStream_t st)
{
    int blocks = 0;
    cudaError_t e = bwd_call(p, partial, &blocks, false, st);
    if (e != cudaSuccess || (!p.grad_weight && !p.grad_bias))
        return e;
    return launch_pdl(layer_params_kernel, dim3((2 * p.dim + 31) / 32), dim3(32, 32), 0, st, partial, blocks, p.dim, p.grad_weight,
                      p.grad_bias);
}

}  // namespace csa
