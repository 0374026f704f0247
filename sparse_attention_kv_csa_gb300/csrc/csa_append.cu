// Rows appended to a paged cache with the position rotation on the way, and queries (or any heads) rotated.
//
// A row is [plain | part]; the part's columns are pairs (a, b), neighbours or half the part apart, each turned by its angle:
//
//   a' = a cos - b sin,  b' = a sin + b cos          (backwards: sin negated)
//
// in fp32 with one rounding, cosines and sines read from a table in fp32 (a row a position, cosines then sines), because an
// angle of a far position needs more than 32 bits before it is reduced.  8-bit rows: scale = max |y| / 448 over the row.
//
// Bound by latency: position, then the table's row, then the products.  A warp has a row in registers, 16 bytes a lane at a time;
// the partner of a vector half a part away is read again (it comes from L1).  Heads: a thread has a vector (or the two that
// belong together) of four heads, so that four loads are under way.  65543 rows of 512 to 8 bits 33.3 us (floor 17.5), the heads of 4099
// tokens, 64 of 64 columns each, 14.1 (10.1): no unit is full in either (DRAM 31% and 25%, issue 56% and 51%), with 43% of the
// warps resident at 54 and 52 registers; 64 rows and their queries 2.6 us.
#include "csa_norm.cuh"

namespace csa {
namespace {

constexpr int kThreads = 256;
constexpr int kHeadsAThread = 4;

// Cosines and sines of pairs [i, i + N) of a position, NaN where the table has no such position.  With N > 1 i, the table's rows
// and its base are whole vectors of min(N, 4) floats.
template <int N> __device__ __forceinline__ void angles(const TurnParams &p, int position, int i, float (&cos)[N], float (&sin)[N])
{
    const bool have = position >= 0 && position < p.n_positions;
    const float *row = p.rotation + (int64_t)(have ? position : 0) * 2 * p.half + i;
    auto get = [&](const float *at, float (&v)[N]) {
        if constexpr (N >= 4) {
#pragma unroll
            for (int k = 0; k < N; k += 4) {
                const float4 f = __ldg(reinterpret_cast<const float4 *>(at + k));
                v[k] = f.x, v[k + 1] = f.y, v[k + 2] = f.z, v[k + 3] = f.w;
            }
        } else if constexpr (N == 2) {
            const float2 f = __ldg(reinterpret_cast<const float2 *>(at));
            v[0] = f.x, v[1] = f.y;
        } else {
            v[0] = __ldg(at);
        }
    };
    if (p.n_positions > 0) {
        get(row, cos);
        get(row + p.half, sin);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        cos[k] = have ? cos[k] : __int_as_float(0x7fffffff);
        sin[k] = have ? (p.inverse ? -sin[k] : sin[k]) : __int_as_float(0x7fffffff);
    }
}

// a cos - b sin and a sin + b cos
__device__ __forceinline__ float2 turn(float a, float b, float cos, float sin)
{
    return make_float2(fmaf(a, cos, -(b * sin)), fmaf(a, sin, b * cos));
}

template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> read(const T *p) { return *reinterpret_cast<const Pack<T, VEC> *>(p); }

// VEC: elements of a vector (16 bytes), or 1; NV: vectors a lane.  Everything that does not hang on another load is read before
// anything is used: a row is some microsecond of latency, and a row's own loads are all that a warp has under way.
template <typename T, bool BITS8, int VEC, int NV> __device__ __forceinline__ void append_row(const AppendParams &p, int64_t row)
{
    const int lane = threadIdx.x & 31, half = p.turn.half, width = p.plain_dim + 2 * half;
    const T *plain = static_cast<const T *>(p.plain) + row * p.plain_stride, *part = static_cast<const T *>(p.part) + row * p.part_stride;
    const int64_t to = __ldg(p.slots + row);
    const int position = __ldg(p.positions + row);
    // the vector of the part that lane's vector i is turned with, when pairs are half the part apart
    auto partner = [&](int j) { return j < half ? j + half : j - half; };
    Pack<T, VEC> in[NV], with[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * 32 + lane) * VEC, j = c - p.plain_dim;
        if (c < width) {
            in[i] = read<T, VEC>(j < 0 ? plain + c : part + j);
            if (j >= 0 && (VEC == 1 || !p.turn.interleaved))
                with[i] = read<T, VEC>(part + (p.turn.interleaved ? j ^ 1 : partner(j)));
        }
    }
    if (to < 0 || to >= p.n_slots)
        return;
    float v[NV][VEC];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * 32 + lane) * VEC, j = c - p.plain_dim;
        if (c >= width)
            continue;
        unpack(in[i], v[i]);
        if (j >= 0) {
            if (VEC > 1 && p.turn.interleaved) {
                if constexpr (VEC > 1) {
                    float cos[VEC / 2], sin[VEC / 2];
                    angles(p.turn, position, j / 2, cos, sin);
#pragma unroll
                    for (int k = 0; k < VEC / 2; ++k) {
                        const float2 t = turn(v[i][2 * k], v[i][2 * k + 1], cos[k], sin[k]);
                        v[i][2 * k] = t.x;
                        v[i][2 * k + 1] = t.y;
                    }
                }
            } else {
                const bool upper = p.turn.interleaved ? j & 1 : j >= half;
                float u[VEC], cos[VEC], sin[VEC];
                unpack(with[i], u);
                angles(p.turn, position, p.turn.interleaved ? j / 2 : upper ? j - half : j, cos, sin);
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    v[i][k] = upper ? turn(u[k], v[i][k], cos[k], sin[k]).y : turn(v[i][k], u[k], cos[k], sin[k]).x;
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
template <typename T, int VEC, bool NEIGHBOURS> __device__ __forceinline__ void turn_heads(const TurnParams &p, int64_t block)
{
    constexpr bool kOne = VEC > 1 && NEIGHBOURS;  // a and b lie in one vector
    constexpr int N = kOne ? VEC / 2 : VEC;       // pairs of a unit
    const int units = p.half / N;
    const int rows = units < kThreads ? kThreads / units : 1;  // heads side by side (a part of more units than threads takes several turns)
    const int64_t end = p.n_tokens * p.n_heads;
    for (int first = 0; first < units; first += kThreads) {
        const int u = first + (units > kThreads ? (int)threadIdx.x : (int)threadIdx.x % units);
        const int sub = units > kThreads ? 0 : (int)threadIdx.x / units;
        if (u >= units || sub >= rows)
            continue;
        const int at_a = NEIGHBOURS ? 2 * N * u : N * u, at_b = NEIGHBOURS ? 2 * u + 1 : N * u + p.half;
        Pack<T, VEC> a[kHeadsAThread], b[kHeadsAThread];
        int position[kHeadsAThread];
        int64_t to[kHeadsAThread];
#pragma unroll
        for (int k = 0; k < kHeadsAThread; ++k) {
            const int64_t row = (block * kHeadsAThread + k) * rows + sub;
            to[k] = -1;
            if (row < end) {
                const uint32_t token = p.by_heads.quotient((uint32_t)row), head = (uint32_t)row - token * (uint32_t)p.n_heads;
                position[k] = __ldg(p.positions + token);
                to[k] = (int64_t)token * p.out_token_stride + (int64_t)head * p.out_head_stride;
                const T *src = static_cast<const T *>(p.x) + (int64_t)token * p.x_token_stride + (int64_t)head * p.x_head_stride;
                a[k] = read<T, VEC>(src + at_a);
                if (!kOne)
                    b[k] = read<T, VEC>(src + at_b);
            }
        }
#pragma unroll
        for (int k = 0; k < kHeadsAThread; ++k) {
            if (to[k] < 0)
                continue;
            T *dst = static_cast<T *>(p.out) + to[k];
            float x[VEC], cos[N], sin[N];
            angles(p, position[k], N * u, cos, sin);
            unpack(a[k], x);
            if constexpr (kOne) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float2 t = turn(x[2 * i], x[2 * i + 1], cos[i], sin[i]);
                    x[2 * i] = t.x;
                    x[2 * i + 1] = t.y;
                }
            } else {
                float y[VEC];
                unpack(b[k], y);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float2 t = turn(x[i], y[i], cos[i], sin[i]);
                    x[i] = t.x;
                    y[i] = t.y;
                }
                store<T, VEC>(dst + at_b, pack<T, VEC>(y));
            }
            store<T, VEC>(dst + at_a, pack<T, VEC>(x));
        }
    }
}

enum Heads { kNone, kScalar, kHalves, kNeighbours };  // heads to turn: none, pair by pair, in vectors of either form

// The first blocks take rows (NV 0: there are none), the others heads.  Forms apart, so that rows alone or heads alone do not run
// with the registers of both (65543 rows of 512: 54 registers a thread against 92).
template <typename T, bool BITS8, int VEC, int NV, Heads HEADS>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p, int row_blocks)
{
    constexpr int V = 16 / sizeof(T);
    pdl_wait();
    pdl_trigger();
    if constexpr (NV > 0)
        if (blockIdx.x < row_blocks) {
            const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
            if (row < p.n_rows)
                append_row<T, BITS8, VEC, NV>(p, row);
            return;
        }
    if constexpr (HEADS == kScalar) {
        if (p.turn.interleaved)
            turn_heads<T, 1, true>(p.turn, blockIdx.x - row_blocks);
        else
            turn_heads<T, 1, false>(p.turn, blockIdx.x - row_blocks);
    } else if constexpr (HEADS != kNone) {
        turn_heads<T, V, HEADS == kNeighbours>(p.turn, blockIdx.x - row_blocks);
    }
}

template <typename T, bool BITS8, int VEC, int NV, Heads HEADS> cudaError_t go(const AppendParams &p, cudaStream_t st)
{
    constexpr int N = HEADS == kScalar ? 1 : HEADS == kNeighbours ? 8 / (int)sizeof(T) : 16 / (int)sizeof(T);
    const int64_t row_blocks = (p.n_rows + kThreads / 32 - 1) / (kThreads / 32);
    const int units = p.turn.half / N;
    const int64_t rows = (int64_t)(units < kThreads ? kThreads / units : 1) * kHeadsAThread;
    const int64_t heads = HEADS == kNone ? 0 : p.turn.n_tokens * p.turn.n_heads;
    return launch_pdl(append_kernel<T, BITS8, VEC, NV, HEADS>, dim3((unsigned)(row_blocks + (heads + rows - 1) / rows)), dim3(kThreads), 0, st,
                      p, (int)row_blocks);
}

template <typename T, bool BITS8, int VEC, int NV> cudaError_t go_heads(const AppendParams &p, Heads heads, cudaStream_t st)
{
    if constexpr (NV > 0)
        if (heads == kNone)
            return go<T, BITS8, VEC, NV, kNone>(p, st);
    return heads == kScalar     ? go<T, BITS8, VEC, NV, kScalar>(p, st)
           : heads == kHalves ? go<T, BITS8, VEC, NV, kHalves>(p, st)
                              : go<T, BITS8, VEC, NV, kNeighbours>(p, st);
}

template <typename T, bool BITS8> cudaError_t go_rows(const AppendParams &p, bool vectors, Heads heads, cudaStream_t st)
{
    constexpr int V = 16 / sizeof(T);
    const int width = p.plain_dim + 2 * p.turn.half;
    if (!vectors)
        return go_heads<T, BITS8, 1, 32>(p, heads, st);
    if (width <= 32 * V) return go_heads<T, BITS8, V, 1>(p, heads, st);
    if (width <= 64 * V) return go_heads<T, BITS8, V, 2>(p, heads, st);
    if (width <= 96 * V) return go_heads<T, BITS8, V, 3>(p, heads, st);
    if constexpr (V == 4)  // (1024 columns of 16 bits are 128 vectors)
        if (width > 128 * V) return go_heads<T, BITS8, V, 8>(p, heads, st);
    return go_heads<T, BITS8, V, 4>(p, heads, st);
}

template <typename T> cudaError_t go_type(const AppendParams &p, cudaStream_t st)
{
    constexpr int v = 16 / sizeof(T);
    const TurnParams &t = p.turn;
    // whole vectors of pairs, and of their angles
    const bool pairs = (t.interleaved ? 2 * t.half % v == 0 : t.half % v == 0) && t.half % 4 == 0 && on(t.rotation, 16);
    const bool in_vectors = pairs && on(t.x, 16) && on(t.out, 16) && t.x_token_stride % v == 0 && t.x_head_stride % v == 0 &&
                            t.out_token_stride % v == 0 && t.out_head_stride % v == 0;
    const Heads heads = t.n_tokens == 0 ? kNone : !in_vectors ? kScalar : t.interleaved ? kNeighbours : kHalves;
    if (p.n_rows == 0)
        return go_heads<T, false, v, 0>(p, heads, st);
    const bool vectors = pairs && p.plain_dim % v == 0 && (p.plain_dim == 0 || (on(p.plain, 16) && p.plain_stride % v == 0)) &&
                         on(p.part, 16) && p.part_stride % v == 0 && p.out_stride % v == 0 && on(p.out, v * elem_bytes(p.out_dtype));
    return p.out_dtype == CSA_DTYPE_E4M3 ? go_rows<T, true>(p, vectors, heads, st) : go_rows<T, false>(p, vectors, heads, st);
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
