// Rows appended to a paged cache with the position rotation on the way, and queries (or any heads) rotated.
//
// A row is [plain | part]; the part's columns are pairs (a, b), neighbours or half the part apart, each turned by its angle:
//
//   a' = a cos - b sin,  b' = a sin + b cos          (backwards: sin negated)
//
// in fp32 with one rounding, cosines and sines read from a table in fp32 (a row a position, cosines then sines), because an
// angle of a far position needs more than 32 bits before it is reduced.  8-bit rows: scale = max |y| / 448 over the row.
//
// Bound by DRAM for many rows and by latency for few: position, then the table's row, then the products.  A warp has a row in
// registers, 16 bytes a lane at a time; the partner of a vector half a part away is read again (it comes from L1).  Heads: a
// thread has a vector (or the two that belong together) of four heads, so that four loads are under way.
#include "csa_norm.cuh"

namespace csa {
namespace {

constexpr int kThreads = 256;
constexpr int kHeadsAThread = 4;

// Cosines and sines of pairs [i, i + N) of a position, NaN where the table has no such position.
template <int N> __device__ __forceinline__ void angles(const TurnParams &p, int position, int i, float (&cos)[N], float (&sin)[N])
{
    const bool have = position >= 0 && position < p.n_positions;
    const float *row = p.rotation + (int64_t)(have ? position : 0) * 2 * p.half;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        cos[k] = have ? __ldg(row + i + k) : __int_as_float(0x7fffffff);
        sin[k] = have ? __ldg(row + p.half + i + k) : __int_as_float(0x7fffffff);
    }
    if (p.inverse)
#pragma unroll
        for (int k = 0; k < N; ++k)
            sin[k] = -sin[k];
}

template <typename T, int VEC> __device__ __forceinline__ void read(const T *p, float (&v)[VEC])
{
    const Pack<T, VEC> a = *reinterpret_cast<const Pack<T, VEC> *>(p);
    unpack(a, v);
}

// VEC: elements of a vector (16 bytes), or 1; NV: vectors a lane
template <typename T, bool BITS8, int VEC, int NV> __device__ void append_row(const AppendParams &p, int64_t row)
{
    const int lane = threadIdx.x & 31, half = p.turn.half, width = p.plain_dim + 2 * half;
    const int64_t to = __ldg(p.slots + row);
    if (to < 0 || to >= p.n_slots)
        return;
    const int position = __ldg(p.positions + row);
    const T *plain = static_cast<const T *>(p.plain) + row * p.plain_stride, *part = static_cast<const T *>(p.part) + row * p.part_stride;
    float v[NV][VEC];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * 32 + lane) * VEC, j = c - p.plain_dim;
        if (c >= width)
            continue;
        if (j < 0) {
            read<T, VEC>(plain + c, v[i]);
        } else {
            read<T, VEC>(part + j, v[i]);
            if (p.turn.interleaved) {
                if constexpr (VEC > 1) {
                    float cos[VEC / 2], sin[VEC / 2];
                    angles(p.turn, position, j / 2, cos, sin);
#pragma unroll
                    for (int k = 0; k < VEC / 2; ++k) {
                        const float a = v[i][2 * k], b = v[i][2 * k + 1];
                        v[i][2 * k] = a * cos[k] - b * sin[k];
                        v[i][2 * k + 1] = a * sin[k] + b * cos[k];
                    }
                } else {
                    float cos[1], sin[1];
                    angles(p.turn, position, j / 2, cos, sin);
                    const float u = Elem<T>::to(part[j ^ 1]);
                    v[i][0] = j & 1 ? u * sin[0] + v[i][0] * cos[0] : v[i][0] * cos[0] - u * sin[0];
                }
            } else {
                const bool upper = j >= half;
                const int pair = upper ? j - half : j;
                float u[VEC], cos[VEC], sin[VEC];
                read<T, VEC>(part + (upper ? pair : pair + half), u);
                angles(p.turn, position, pair, cos, sin);
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    v[i][k] = upper ? u[k] * sin[k] + v[i][k] * cos[k] : v[i][k] * cos[k] - u[k] * sin[k];
            }
        }
        if constexpr (BITS8)
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                amax = max_nan(amax, fabsf(v[i][k]));
    }
    if constexpr (!BITS8) {
        T *out = static_cast<T *>(p.out) + to * p.out_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * 32 + lane) * VEC;
            if (c < width)
                store<T, VEC>(out + c, pack<T, VEC>(v[i]));
        }
    } else {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            amax = max_nan(amax, __shfl_xor_sync(~0u, amax, o));
        const float scale = amax / kE4m3Max;
        // y / scale within two roundings of fp32, far below e4m3's half step; a row of zeros keeps scale 0; a scale whose
        // reciprocal would overflow divides instead
        const bool tiny = scale < 1e-37f;
        const float inv = scale > 0.0f && !tiny ? 1.0f / scale : 1.0f;
        __nv_fp8_storage_t *out = static_cast<__nv_fp8_storage_t *>(p.out) + to * p.out_stride;
        if (lane == 0)
            p.scales[to] = scale;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * 32 + lane) * VEC;
            if (c >= width)
                continue;
            if (tiny && scale > 0.0f)
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    v[i][k] /= scale;
            scale_by(v[i], inv);
            Pack<__nv_fp8_storage_t, VEC> o;
            if constexpr (VEC > 1) {
#pragma unroll
                for (int k = 0; k < VEC; k += 2) {
                    const __nv_fp8x2_storage_t two = __nv_cvt_float2_to_fp8x2(make_float2(v[i][k], v[i][k + 1]), __NV_SATFINITE, __NV_E4M3);
                    memcpy(&o.v[k], &two, 2);
                }
            } else {
                o.v[0] = __nv_cvt_float_to_fp8(v[i][0], __NV_SATFINITE, __NV_E4M3);
            }
            store<__nv_fp8_storage_t, VEC>(out + c, o);
        }
    }
}

// Heads: unit u of a head is its vector u (pairs of neighbours), or the vectors u and u + units (pairs half a part apart); with
// VEC 1 a unit is a pair.
template <typename T, int VEC> __device__ void turn_heads(const TurnParams &p, int64_t block)
{
    constexpr int N = VEC;  // values of each of a and b in the halves' form; neighbours have N / 2 pairs
    const int units = VEC == 1 ? p.half : p.interleaved ? 2 * p.half / VEC : p.half / VEC;
    const int rows = kThreads / units > 0 ? kThreads / units : 1;  // (a part of more units than threads takes several turns)
    for (int first = 0; first < units; first += kThreads) {
        const int u = first + (units > kThreads ? (int)threadIdx.x : (int)threadIdx.x % units);
        const int sub = units > kThreads ? 0 : (int)threadIdx.x / units;
        if (u >= units || sub >= rows)
            continue;
        const int at_a = VEC == 1 && p.interleaved ? 2 * u : u * VEC, at_b = VEC == 1 && p.interleaved ? 2 * u + 1 : u * VEC + p.half;
        const int pair = VEC > 1 && p.interleaved ? u * VEC / 2 : u * VEC;
        float a[kHeadsAThread][N], b[kHeadsAThread][N];
        int position[kHeadsAThread];
        int64_t row[kHeadsAThread];
        const bool neighbours = VEC > 1 && p.interleaved;
#pragma unroll
        for (int k = 0; k < kHeadsAThread; ++k) {
            row[k] = (block * kHeadsAThread + k) * rows + sub;
            if (row[k] < p.n_tokens * p.n_heads) {
                const uint32_t token = p.by_heads.quotient((uint32_t)row[k]), head = p.by_heads.remainder((uint32_t)row[k]);
                position[k] = __ldg(p.positions + token);
                const T *src = static_cast<const T *>(p.x) + (int64_t)token * p.x_token_stride + (int64_t)head * p.x_head_stride;
                read<T, VEC>(src + at_a, a[k]);
                if (!neighbours)
                    read<T, VEC>(src + at_b, b[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < kHeadsAThread; ++k) {
            if (row[k] >= p.n_tokens * p.n_heads)
                continue;
            const uint32_t token = p.by_heads.quotient((uint32_t)row[k]), head = p.by_heads.remainder((uint32_t)row[k]);
            T *dst = static_cast<T *>(p.out) + (int64_t)token * p.out_token_stride + (int64_t)head * p.out_head_stride;
            if (neighbours) {
                if constexpr (VEC > 1) {
                    float cos[VEC / 2], sin[VEC / 2];
                    angles(p, position[k], pair, cos, sin);
#pragma unroll
                    for (int i = 0; i < VEC / 2; ++i) {
                        const float x = a[k][2 * i], y = a[k][2 * i + 1];
                        a[k][2 * i] = x * cos[i] - y * sin[i];
                        a[k][2 * i + 1] = x * sin[i] + y * cos[i];
                    }
                    store<T, VEC>(dst + at_a, pack<T, VEC>(a[k]));
                }
            } else {
                float cos[N], sin[N];
                angles(p, position[k], pair, cos, sin);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float x = a[k][i], y = b[k][i];
                    a[k][i] = x * cos[i] - y * sin[i];
                    b[k][i] = x * sin[i] + y * cos[i];
                }
                store<T, VEC>(dst + at_a, pack<T, VEC>(a[k]));
                store<T, VEC>(dst + at_b, pack<T, VEC>(b[k]));
            }
        }
    }
}

// The first blocks take rows, the others heads.  VEC, NV: of the rows; HVEC: of the heads.
template <typename T, bool BITS8, int VEC, int NV, int HVEC>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p, int row_blocks)
{
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x < row_blocks) {
        const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
        if (row < p.n_rows)
            append_row<T, BITS8, VEC, NV>(p, row);
    } else {
        turn_heads<T, HVEC>(p.turn, blockIdx.x - row_blocks);
    }
}

template <typename T, bool BITS8, int VEC, int NV, int HVEC> cudaError_t go(const AppendParams &p, cudaStream_t st)
{
    const int row_blocks = (int)((p.n_rows + kThreads / 32 - 1) / (kThreads / 32));
    const int units = HVEC == 1 ? p.turn.half : p.turn.interleaved ? 2 * p.turn.half / HVEC : p.turn.half / HVEC;
    const int64_t rows = (int64_t)(kThreads / units > 0 ? kThreads / units : 1) * kHeadsAThread;
    const int64_t heads = p.turn.n_tokens * p.turn.n_heads;
    return launch_pdl(append_kernel<T, BITS8, VEC, NV, HVEC>, dim3((unsigned)(row_blocks + (heads + rows - 1) / rows)), dim3(kThreads), 0, st,
                      p, row_blocks);
}

template <typename T, bool BITS8, int VEC, int NV> cudaError_t go_heads(const AppendParams &p, bool head_vectors, cudaStream_t st)
{
    return head_vectors ? go<T, BITS8, VEC, NV, 16 / sizeof(T)>(p, st) : go<T, BITS8, VEC, NV, 1>(p, st);
}

template <typename T, bool BITS8> cudaError_t go_rows(const AppendParams &p, bool row_vectors, bool head_vectors, cudaStream_t st)
{
    constexpr int V = 16 / sizeof(T);
    const int width = p.n_rows ? p.plain_dim + 2 * p.turn.half : 1;
    if (row_vectors) {
        if (width <= 32 * V) return go_heads<T, BITS8, V, 1>(p, head_vectors, st);
        if (width <= 64 * V) return go_heads<T, BITS8, V, 2>(p, head_vectors, st);
        if (width <= 96 * V) return go_heads<T, BITS8, V, 3>(p, head_vectors, st);
        if (V == 8 || width <= 128 * V) return go_heads<T, BITS8, V, 4>(p, head_vectors, st);
        return go_heads<T, BITS8, V, 8>(p, head_vectors, st);
    }
    return go_heads<T, BITS8, 1, 32>(p, head_vectors, st);
}

template <typename T> cudaError_t go_type(const AppendParams &p, cudaStream_t st)
{
    constexpr int v = 16 / sizeof(T);
    const TurnParams &t = p.turn;
    const bool pairs = t.interleaved ? 2 * t.half % v == 0 : t.half % v == 0;
    const bool rows = p.n_rows == 0 || (pairs && p.plain_dim % v == 0 && (p.plain_dim == 0 || (on(p.plain, 16) && p.plain_stride % v == 0)) &&
                                        on(p.part, 16) && p.part_stride % v == 0 && p.out_stride % v == 0 &&
                                        on(p.out, v * elem_bytes(p.out_dtype)));
    const bool heads = t.n_tokens == 0 || (pairs && on(t.x, 16) && on(t.out, 16) && t.x_token_stride % v == 0 && t.x_head_stride % v == 0 &&
                                           t.out_token_stride % v == 0 && t.out_head_stride % v == 0);
    return p.out_dtype == CSA_DTYPE_E4M3 ? go_rows<T, true>(p, rows, heads, st) : go_rows<T, false>(p, rows, heads, st);
}

}  // namespace

cudaError_t launch_append(const AppendParams &p, cudaStream_t st)
{
    switch (p.dtype) {
    case CSA_DTYPE_BF16: return go_type<__nv_bfloat16>(p, st);
    case CSA_DTYPE_F16: return go_type<__half>(p, st);
    default: return go_type<float>(p, st);
    }
}

}  // namespace csa
