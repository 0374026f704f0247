// The norm's forward (see csa_norm.cuh).
#include "csa_norm.cuh"

namespace csa {
namespace {

// Every thread of a block runs the same number of rows (idle teams take no row), so the barriers above are uniform.
template <typename T, typename OUT, int VEC, int TEAM, int NV, bool STAGED>
__global__ void __launch_bounds__(TEAM < 128 ? 128 : TEAM)
norm_fwd_kernel(const NormFwdParams p)
{
    constexpr int kThreads = TEAM < 128 ? 128 : TEAM;
    constexpr int kTeams = kThreads / TEAM;
    constexpr bool kBits8 = sizeof(OUT) == 1;
    __shared__ float buf[4][kThreads / 32];
    __shared__ uint64_t all_full[kTeams * kMaxRing];
    extern __shared__ __align__(128) uint8_t ring_mem[];
    const int t = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
    uint64_t *full = all_full + team * kMaxRing;
    const int arrays = p.residual ? 2 : 1, row_bytes = p.dim * (int)sizeof(T);
    const Ring ring{ring_mem + team * p.stages * arrays * row_bytes, full, p.stages, row_bytes, arrays, p.status};
    if (STAGED)
        ring.init(t == 0);
    pdl_wait();
    pdl_trigger();
    const T *x = static_cast<const T *>(p.x), *res = static_cast<const T *>(p.residual);
    float w[NV][VEC];
    bool odd_weight = false;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const int c = (i * TEAM + t) * VEC + k;
            w[i][k] = c < p.dim ? (p.weight ? __ldg(p.weight + c) : 1.0f) : 0.0f;
            odd_weight |= !(fabsf(w[i][k]) < INFINITY);
        }
    // 128 columns lie in 128 / VEC neighbouring lanes; the host takes that form with whole vectors only
    const bool grouped = VEC * sizeof(T) == 16 && p.scale_group == 128;
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
            // (16394 rows of 4100: 303 us with, 140 without)
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
        float2 ss2 = splat(0.0f);
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
                ss2 = dot_add(h[i], h[i], ss2);
            } else {
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    h[i][k] = 0.0f;
            }
        }
        fetch(row + step);
        const float ss = team_reduce<TEAM, false>(ss2.x + ss2.y, buf[it & 1]);
        if (STAGED) {
            // the sum's barrier: the whole team has read the stage
            if (TEAM <= 32)
                __syncwarp();
            if (t == 0 && at.ok)
                refill(row + ring.stages * step, at.stage);
            ring.next(at);
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
        // The plain maximum drops NaN.  A NaN among the y needs a sum that is not finite, a zero row without eps (0 times
        // an infinite rstd) or a weight that is not finite.
        const bool odd = !(ss < INFINITY) || !(rstd < INFINITY) || odd_weight;
        auto magnitude = [&](int i, float m) {
            if (odd) {
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    m = max_nan(m, fabsf(h[i][k]));
            } else {
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    m = fmaxf(m, fabsf(h[i][k]));
            }
            return m;
        };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            scale_by(h[i], rstd);
            scale_by(h[i], w[i]);
            if (kBits8 && !grouped)
                amax = magnitude(i, amax);
        }
        if (kBits8 && !grouped)
            amax = team_reduce<TEAM, true>(amax, buf[2 + (it & 1)]);
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
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TEAM + t) * VEC;
                if (grouped) {
                    amax = magnitude(i, 0.0f);
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
                    scale_by(h[i], inv);
                    if constexpr (VEC > 1) {
#pragma unroll
                        for (int k = 0; k < VEC; k += 2) {
                            const __nv_fp8x2_storage_t two =
                                __nv_cvt_float2_to_fp8x2(make_float2(h[i][k], h[i][k + 1]), __NV_SATFINITE, __NV_E4M3);
                            memcpy(&o.v[k], &two, 2);
                        }
                    } else {
                        o.v[0] = __nv_cvt_float_to_fp8(h[i][0], __NV_SATFINITE, __NV_E4M3);
                    }
                    store<__nv_fp8_storage_t, VEC>(reinterpret_cast<__nv_fp8_storage_t *>(out) + c, o);
                    if (grouped ? (c & 127) == 0 : c == 0)
                        p.scales[to * (grouped ? p.dim / 128 : 1) + (grouped ? c / 128 : 0)] = scale;
                }
            }
        }
    }
}

template <typename T, typename OUT, int VEC, int TEAM, int NV>
cudaError_t fwd_go(NormFwdParams p, cudaStream_t st)
{
    constexpr int threads = TEAM < 128 ? 128 : TEAM;
    auto k = norm_fwd_kernel<T, OUT, VEC, TEAM, NV, false>;
    size_t smem = 0;
    int grid = 0;
    cudaError_t e = norm_plan(k, norm_fwd_kernel<T, OUT, VEC, TEAM, NV, VEC * sizeof(T) == 16>, threads, threads / TEAM,
                              p.dim * (int)sizeof(T), p.residual ? 2 : 1, kRingForward, p.n_rows, &k, &p.stages, &smem, &grid);
    return e == cudaSuccess ? launch_pdl(k, dim3(grid), dim3(threads), smem, st, p) : e;
}

template <typename T, typename OUT> cudaError_t fwd_size(const NormFwdParams &p, int vec, cudaStream_t st)
{
    constexpr int V = 16 / sizeof(T);
    if (vec == V) {
        const int words = p.dim / V;
        // Many narrow rows: two a warp, which halves what a row costs besides its elements (200000 rows of 128 46 us with
        // one, 29 with two; 131288 of 512 to 8 bits 66 and 64); few: one, which is done sooner (8256 of 512 6.5 and 7.7).
        // Types of 16 bits alone: half a warp's words have to hold a group of 128 columns.
        if constexpr (V == 8) {
            if (words <= 64 && p.n_rows >= 32768) {
                if (words <= 16) return fwd_go<T, OUT, V, 16, 1>(p, st);
                if (words <= 32) return fwd_go<T, OUT, V, 16, 2>(p, st);
                return fwd_go<T, OUT, V, 16, 4>(p, st);
            }
        }
        if (words <= 32) return fwd_go<T, OUT, V, 32, 1>(p, st);
        if (words <= 64) return fwd_go<T, OUT, V, 32, 2>(p, st);
        // (200000 rows of 576 to 8 bits: 170 us with four words a thread, 152 with three)
        if (words <= 96) return fwd_go<T, OUT, V, 32, 3>(p, st);
        if (words <= 128) return fwd_go<T, OUT, V, 32, 4>(p, st);
        if (words <= 256) return fwd_go<T, OUT, V, 128, 2>(p, st);
        if (words <= 512) return fwd_go<T, OUT, V, 128, 4>(p, st);
        if (words <= 1024) return fwd_go<T, OUT, V, 256, 4>(p, st);
        if constexpr (V == 4)  // (16384 columns of 16 bits are 2048 words)
            if (words > 2048) return fwd_go<T, OUT, V, 1024, 4>(p, st);
        return fwd_go<T, OUT, V, 512, 4>(p, st);
    }
    if constexpr (sizeof(T) == 2)
        if (vec == 2) {
            if (p.dim <= 512) return fwd_go<T, OUT, 2, 32, 8>(p, st);
            if (p.dim <= 1024) return fwd_go<T, OUT, 2, 64, 8>(p, st);
            if (p.dim <= 2048) return fwd_go<T, OUT, 2, 128, 8>(p, st);
            if (p.dim <= 4096) return fwd_go<T, OUT, 2, 128, 16>(p, st);
            if (p.dim <= 8192) return fwd_go<T, OUT, 2, 256, 16>(p, st);
            return fwd_go<T, OUT, 2, 512, 16>(p, st);
        }
    if (p.dim <= 512) return fwd_go<T, OUT, 1, 32, 16>(p, st);
    if (p.dim <= 1024) return fwd_go<T, OUT, 1, 64, 16>(p, st);
    if (p.dim <= 2048) return fwd_go<T, OUT, 1, 128, 16>(p, st);
    if (p.dim <= 4096) return fwd_go<T, OUT, 1, 256, 16>(p, st);
    if (p.dim <= 8192) return fwd_go<T, OUT, 1, 512, 16>(p, st);
    return fwd_go<T, OUT, 1, 1024, 16>(p, st);
}

int norm_fwd_vector(const NormFwdParams &p)
{
    return widest(p.dtype, [&](int v) {
        const int b = v * elem_bytes(p.dtype);
        return p.dim % v == 0 && p.x_stride % v == 0 && on(p.x, b) &&
               (!p.residual || (p.residual_stride % v == 0 && on(p.residual, b))) && on(p.residual_out, b) &&
               p.out_stride % v == 0 && on(p.out, v * elem_bytes(p.out_dtype));
    });
}

}  // namespace

bool norm_fwd_whole_vectors(const NormFwdParams &p) { return norm_fwd_vector(p) == 16 / elem_bytes(p.dtype); }

cudaError_t launch_norm_fwd(const NormFwdParams &p, cudaStream_t st)
{
    const int vec = norm_fwd_vector(p);
    const bool bits8 = p.out_dtype == CSA_DTYPE_E4M3;
    switch (p.dtype) {
    case CSA_DTYPE_BF16:
        return bits8 ? fwd_size<__nv_bfloat16, __nv_fp8_e4m3>(p, vec, st) : fwd_size<__nv_bfloat16, __nv_bfloat16>(p, vec, st);
    case CSA_DTYPE_F16:
        return bits8 ? fwd_size<__half, __nv_fp8_e4m3>(p, vec, st) : fwd_size<__half, __half>(p, vec, st);
    default:
        return bits8 ? fwd_size<float, __nv_fp8_e4m3>(p, vec, st) : fwd_size<float, float>(p, vec, st);
    }
}

}  // namespace csa
