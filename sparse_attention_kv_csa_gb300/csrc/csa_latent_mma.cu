// Attention over a paged cache of shared latent rows on the tensor cores (tcgen05).
//
// The query rows of a request are its (token, head) pairs, in order; all of them read the same cache rows.  An item is
// 64 such rows.  For each tile of 32 cache rows:
//
//   S = Q K^T          64 x 32, K = head_dim: both operands K-major in shared memory
//   P = exp2(S f - m)  f = scale log2 e, m the row's reference; l += sum P; P to bf16 in shared memory
//   O = O + P V        64 x v_dim, K = 32 cache rows; V is the K tile itself, read with its rows along K
//
// so a cache row is fetched once and used for both products.  m is raised (O and l scaled down) only when a logit
// exceeds it by 2^8: P stays below 2^8, which bf16 and the fp32 sums hold as well as values below one, and O is
// rarely touched outside the tensor core.
//
// Tensor memory: a 64-row accumulator takes 16 of each 32 lanes, so O (up to 512 columns) has the lower sixteen and
// two S tiles the upper sixteen.  64 query rows, not 128: O of 128 x 512 alone would fill tensor memory, and a K tile
// of 576 columns and 128 query rows would not fit shared memory twice.
//
// Warps: 0-3 exponentials and output (each owns 16 query rows: its quarter of the lanes), 4 issues the MMAs.  bf16
// rows: warp 5 has TMA write whole boxes of rows that lie together in a page, or any four rows at a time where pages
// are small or rows end inside the tile (rows that no query of the item sees read as zeros); warps 6-9 bring the next
// item's queries through registers.  8-bit rows: warps 5-12 bring rows to registers (a tile ahead), widen them to bf16
// (exact) and write the swizzled layout.  Their scale, one a row, multiplies S by column and P before its rounding, so
// it costs no precision.
//
// Work is cut evenly: item i counts one unit for its queries and output and one for each tile; block c takes the units
// [c T / G, (c+1) T / G) of the T units.  Items that cross a cut leave (O, m, l) of their parts in the workspace and a
// second kernel joins them in order.  Nothing else depends on the grid, and no order on timing.
#include <cuda.h>
#include <cuda_fp8.h>

#include "csa_launch.h"
#include "csa_serving_launch.h"
#include "csa_tcgen05.cuh"

namespace csa {
namespace {

constexpr int kTile = 64;                         // query rows of an item
constexpr int kRows = 32;                         // cache rows of a tile
constexpr int kQueryChunk = kTile * 128;          // bytes of 64 columns of an item's queries
constexpr int kChunk = kRows * 128;               // bytes of 64 columns of a tile
constexpr int kSoftWarps = 4;
constexpr int kMmaWarp = 4;
constexpr int kLoadWarps = 8;                     // 8-bit rows
constexpr int kTmaWarp = 5;                       // bf16 rows
constexpr int kQueryWarps = 4;                    // bf16 rows: warps that bring queries
template <bool BITS8> constexpr int kThreadsOf = 32 * (BITS8 ? kSoftWarps + 1 + kLoadWarps : kTmaWarp + 1 + kQueryWarps);
constexpr int kMaxStages = 8;
constexpr float kLog2E = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kRaise = 8.0f;                    // log2 of how far a logit may exceed the reference

struct MmaPlan {
    int nk;           // 64-column chunks of a row
    int stages;
    int blocks;       // G
    int min_units;
    int box_rows;     // rows of a TMA box (a power of two that divides the page), 0: four rows at a time only
    uint32_t tmem_columns;
    size_t smem;
    float *part_o;    // [2 blocks][64][v_dim]
    float2 *part_ml;  // [2 blocks][64]  (m, l)
    int4 *joins;      // [blocks]  (query row, rows, last block, valid): the item that block c is the first of several for
};

struct Shared {
    uint64_t kv_full[kMaxStages], kv_empty[kMaxStages], s_full[2], p_full[2], q_full, q_empty, flags, drained;
    long long sums[16];
    long long total;
    int r, m, off;               // where the block's units begin
    uint32_t tmem;
    alignas(16) float scales[kMaxStages][kRows];
    // rows of the tile that some query sees: 32 bits (bf16 rows), or four bits a byte
    alignas(8) uint8_t valid[kMaxStages][8];
    alignas(4) uint8_t poison[2][kSoftWarps];
};

// What an item is made of.
struct Request {
    int first;    // first token
    int nq;
    int before;   // tokens of the request before its first new one (may be negative)
    int items;
};

__device__ __forceinline__ Request request(const AttnParams &p, int r)
{
    Request q;
    q.first = max(__ldg(p.cu_q + r), 0);
    const int64_t end = min((int64_t)__ldg(p.cu_q + r + 1), p.n_tokens);
    q.nq = (int)max(end - q.first, (int64_t)0);
    q.before = __ldg(p.seq_lens + r) - (__ldg(p.cu_q + r + 1) - q.first);
    q.items = (int)(((int64_t)q.nq * p.n_heads + kTile - 1) / kTile);
    return q;
}

__device__ __forceinline__ int visible(const AttnParams &p, const Request &q, int token)
{
    const int held = q.before + token + 1;
    return held <= 0 ? 0 : min(held / p.ratio, p.width * p.page_size);
}

__device__ __forceinline__ int last_token(const AttnParams &p, const Request &q, int m)
{
    const int64_t row = min((int64_t)(m + 1) * kTile, (int64_t)q.nq * p.n_heads) - 1;
    return (int)(row / p.n_heads);
}

__device__ __forceinline__ int item_tiles(const AttnParams &p, const Request &q, int m)
{
    return (visible(p, q, last_token(p, q, m)) + kRows - 1) / kRows;
}

// The block's segments, walked alike by every role.
struct Walk {
    const AttnParams &p;
    Request q;
    int r, m, off;
    long long left;
    int nt, t0, t1;
    __device__ Walk(const AttnParams &p_, const Shared &s, long long units) : p(p_), r(s.r), m(s.m), off(s.off), left(units)
    {
        if (left > 0)
            q = request(p, r);
    }
    // the next segment: tiles [t0, t1) of item (r, m); nt == 0 (t0 == t1) is an item that sees nothing
    __device__ bool next()
    {
        while (left > 0) {
            while (m >= q.items) {
                if (++r >= p.n_req)
                    return false;
                m = 0;
                q = request(p, r);
            }
            nt = item_tiles(p, q, m);
            const int take = (int)min((long long)(nt + 1 - off), left);
            const bool head = off == 0;
            t0 = max(off - 1, 0);
            t1 = off + take - 1;
            left -= take;
            off = 0;
            ++m;
            if (t1 > t0 || (nt == 0 && head))
                return true;
        }
        return false;
    }
    __device__ int item() const { return m - 1; }
};

__device__ __forceinline__ uint4 zero4() { return make_uint4(0, 0, 0, 0); }

__device__ __forceinline__ bool nonfinite_bf16(uint32_t w)
{
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

__device__ __forceinline__ uint32_t bf16x2_of_e4m3x2(uint32_t two)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    return f2_to_bf16x2(__half22float2(*reinterpret_cast<const __half2 *>(&h)));
}

// Unit cut: block c's first unit.
__device__ __forceinline__ long long cut(long long total, int c, int g) { return total * c / g; }

template <bool BITS8, int NKB>
__global__ void __launch_bounds__(kThreadsOf<BITS8>, 1)
latent_mma_kernel(const AttnParams p, const MmaPlan plan, const __grid_constant__ CUtensorMap boxes,
                  const __grid_constant__ CUtensorMap single, unsigned *status)
{
    constexpr int kThreads = kThreadsOf<BITS8>;
    constexpr int kQueryArrivals = BITS8 ? kLoadWarps : kQueryWarps;
    extern __shared__ uint8_t raw[];
    __shared__ Shared s;
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const int nk = plan.nk, stages = plan.stages;
    // P: rows of 128 bytes, the even tiles' 32 columns in the first half, the odd tiles' in the second
    uint8_t *q_mem = base, *p_mem = q_mem + nk * kQueryChunk, *kv_mem = p_mem + kQueryChunk;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(smem_addr(&s.kv_full[i]), BITS8 ? kLoadWarps : 1);
            mbar_init(smem_addr(&s.kv_empty[i]), 1);
        }
        mbar_init(smem_addr(&s.s_full[0]), 1);
        mbar_init(smem_addr(&s.s_full[1]), 1);
        // (two, by the tile's parity: a warp may be a tile ahead of another)
        mbar_init(smem_addr(&s.p_full[0]), kSoftWarps);
        mbar_init(smem_addr(&s.p_full[1]), kSoftWarps);
        mbar_init(smem_addr(&s.q_full), kQueryArrivals);
        mbar_init(smem_addr(&s.q_empty), 1);
        mbar_init(smem_addr(&s.flags), kSoftWarps);
        mbar_init(smem_addr(&s.drained), 1);
        mbar_init_fence();
    }
    pdl_wait();
    pdl_trigger();
    if (warp == kMmaWarp)
        tmem_alloc(smem_addr(&s.tmem), plan.tmem_columns);

    // ---- where this block's units begin: prefix sums of items over requests (in the space of the tiles), then of
    // units over equal stretches of items, a stretch a thread
    int *items = reinterpret_cast<int *>(base);
    {
        int run = 0;
        int *warp_sum = reinterpret_cast<int *>(s.sums);
        for (int at = 0; at < p.n_req; at += kThreads) {
            const int r = at + tid;
            const int n = r < p.n_req ? request(p, r).items : 0;
            int a = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(~0u, a, o);
                if (lane >= o)
                    a += u;
            }
            if (lane == 31)
                warp_sum[warp] = a;
            __syncthreads();
            int before = run;
            for (int i = 0; i < kThreads / 32; ++i) {
                before += i < warp ? warp_sum[i] : 0;
                run += warp_sum[i];
            }
            if (r < p.n_req)
                items[r] = before + a - n;
            __syncthreads();
        }
        if (tid == 0)
            items[p.n_req] = run;
        __syncthreads();
        const int per = (run + kThreads - 1) / kThreads, lo = min(run, tid * per), hi = min(run, lo + per);
        auto walk = [&](auto &&visit) {
            if (lo >= hi)
                return;
            int r = 0;  // items[r] <= lo < items[r + 1]
            for (int top = p.n_req; top - r > 1;) {
                const int mid = (r + top) >> 1;
                if (items[mid] <= lo)
                    r = mid;
                else
                    top = mid;
            }
            Request q = request(p, r);
            int m = lo - items[r];
            for (int i = lo; i < hi; ++i, ++m) {
                while (m >= q.items) {
                    q = request(p, ++r);
                    m = 0;
                }
                visit(r, m, item_tiles(p, q, m) + 1);
            }
        };
        long long mine = 0;
        walk([&](int, int, int units) { mine += units; });
        long long a = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(~0u, a, o);
            if (lane >= o)
                a += u;
        }
        if (lane == 31)
            s.sums[warp] = a;
        __syncthreads();
        long long before = 0, total = 0;
        for (int i = 0; i < kThreads / 32; ++i) {
            before += i < warp ? s.sums[i] : 0;
            total += s.sums[i];
        }
        const long long first = before + a - mine;
        long long g = total / plan.min_units;
        g = max(1ll, min(g, (long long)plan.blocks));
        const long long from = cut(total, blockIdx.x, (int)g);
        if (blockIdx.x < g && from >= first && from < first + mine) {
            long long at = first;
            walk([&](int r, int m, int units) {
                if (from >= at && from < at + units) {
                    s.r = r;
                    s.m = m;
                    s.off = (int)(from - at);
                }
                at += units;
            });
        }
        if (tid == 0)
            s.total = total;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const long long total = s.total;
    const int g = (int)max(1ll, min(total / plan.min_units, (long long)plan.blocks));
    const int c = blockIdx.x;
    const long long from = cut(total, c, g), units = c < g ? cut(total, c + 1, g) - from : 0;
    const uint32_t tmem = s.tmem;
    bool ok = true;

    if (warp < kSoftWarps) {
        // ------------------------------------------------ exponentials and output
        if (tid == 0)
            plan.joins[c] = make_int4(0, 0, 0, 0);
        const uint32_t my_lanes = tmem + ((uint32_t)(warp * 32) << 16);
        // S: this thread has columns 8 g + 2 (lane % 4) + {0, 1} of rows r0 (x[4g], x[4g + 1]) and r0 + 8
        const int r0 = warp * 16 + lane / 4, cq = 2 * (lane & 3);
        const float f = p.scale * kLog2E;
        int tile = 0;                             // tiles of the block so far
        int flagged = 0;                          // of them, those whose rows were looked through
        long long unit = from;
        Walk w(p, s, units);
        while (ok) {
            const long long left = w.left;
            if (!w.next())
                break;
            unit += left - w.left;  // one past the segment's last unit
            const int item_rows = min(kTile, w.q.nq * p.n_heads - w.item() * kTile);
            const int64_t out_row = (int64_t)w.q.first * p.n_heads + (int64_t)w.item() * kTile;
            auto seen_by = [&](int row) {
                return row < item_rows ? visible(p, w.q, (w.item() * kTile + row) / p.n_heads) : 0;
            };
            const int seen0 = seen_by(r0), seen1 = seen_by(r0 + 8);
            const int all_see = visible(p, w.q, (int)((int64_t)w.item() * kTile / p.n_heads));
            const int end = visible(p, w.q, last_token(p, w.q, w.item()));
            const bool whole = item_rows == kTile;
            float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;  // l: this thread's columns only
            for (int t = w.t0; t < w.t1 && ok; ++t, ++tile) {
                const int st = tile % stages, b = tile & 1;
                // (the loaders' own barrier too: their scales and flags are read below)
                ok = mbar_wait(smem_addr(&s.kv_full[st]), (tile / stages) & 1, status) &&
                     mbar_wait(smem_addr(&s.s_full[b]), (tile >> 1) & 1, status);
                ok = __all_sync(~0u, ok);
                if (!ok)
                    break;
                tc_fence_after();
                float x[16];
                tmem_ld_16x256(my_lanes + (16u << 16) + b * kRows, x);
                tmem_wait_ld();
                float2 rs[4];
                if constexpr (BITS8) {
#pragma unroll
                    for (int g8 = 0; g8 < 4; ++g8)
                        rs[g8] = *reinterpret_cast<const float2 *>(&s.scales[st][8 * g8 + cq]);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    x[i] *= f;
                    if constexpr (BITS8)
                        x[i] *= (i & 1) ? rs[i / 4].y : rs[i / 4].x;
                }
                uint32_t valid;
                if constexpr (BITS8) {
                    const uint64_t v = *reinterpret_cast<const volatile uint64_t *>(s.valid[st]);
                    valid = ~0u;
                    if (v != 0x0f0f0f0f0f0f0f0full) {
                        valid = 0;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            valid |= (uint32_t)(v >> (8 * i) & 0xf) << (4 * i);
                    }
                } else {
                    valid = *reinterpret_cast<const volatile uint32_t *>(s.valid[st]);
                }
                if (!whole || (t + 1) * kRows > all_see || valid != ~0u) {
                    uint32_t poison = 0;
                    if (all_see < end && (t + 1) * kRows > all_see) {
                        // Rows that some queries see and some do not: a weight of zero times an infinity or NaN would
                        // reach the queries that do not, so such a row is cleared, and the queries that see it get NaN.
                        const int row = tid >> 2;
                        uint8_t *mem = kv_mem + st * nk * kChunk + row * 128 + (tid & 3) * 32;
                        bool bad = false;
                        if (t * kRows + row >= all_see && t * kRows + row < end)
                            for (int ch = 0; ch < nk; ++ch)
#pragma unroll
                                for (int u = 0; u < 2; ++u) {
                                    const uint4 v = *reinterpret_cast<const uint4 *>(mem + ch * kChunk + u * 16);
                                    bad |= nonfinite_bf16(v.x) || nonfinite_bf16(v.y) || nonfinite_bf16(v.z) || nonfinite_bf16(v.w);
                                }
                        const uint32_t lanes = __ballot_sync(~0u, bad);
                        if (lanes >> (lane & ~3) & 0xfu)
                            for (int ch = 0; ch < nk; ++ch)
#pragma unroll
                                for (int u = 0; u < 2; ++u)
                                    *reinterpret_cast<uint4 *>(mem + ch * kChunk + u * 16) = zero4();
                        uint32_t bits = 0;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            bits |= (lanes >> (4 * i) & 0xfu) ? 1u << i : 0u;
                        // (two sets: a warp writes one again only after every warp has read it)
                        if (lane == 0) {
                            s.poison[flagged & 1][warp] = (uint8_t)bits;
                            mbar_arrive(smem_addr(&s.flags));
                        }
                        ok = mbar_wait(smem_addr(&s.flags), flagged & 1, status);
                        ok = __all_sync(~0u, ok);
                        if (!ok)
                            break;
                        poison = *reinterpret_cast<const volatile uint32_t *>(s.poison[flagged & 1]) >> cq;
                        ++flagged;
                    }
                    auto mask = [&](int seen) {
                        const int lim = seen - t * kRows;
                        return (valid & (lim <= 0 ? 0u : lim >= 32 ? ~0u : (1u << lim) - 1)) >> cq;
                    };
                    const uint32_t see0 = mask(seen0), see1 = mask(seen1);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int bit = 8 * (i / 4) + (i & 1);
                        if (poison >> bit & 1)
                            x[i] = __int_as_float(0x7fffffff);
                        if (!(((i & 2) ? see1 : see0) >> bit & 1))
                            x[i] = -INFINITY;
                    }
                }
                float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    t0 = fmaxf(t0, fmaxf(x[i], x[i + 1]));
                    t1 = fmaxf(t1, fmaxf(x[i + 2], x[i + 3]));
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    t0 = fmaxf(t0, __shfl_xor_sync(~0u, t0, o));
                    t1 = fmaxf(t1, __shfl_xor_sync(~0u, t1, o));
                }
                const bool up0 = t0 > m0 + kRaise, up1 = t1 > m1 + kRaise;  // (-inf > -inf is false)
                if (__any_sync(~0u, up0 || up1)) {
                    const float d0 = up0 ? exp2_fast(m0 - t0) : 1.0f, d1 = up1 ? exp2_fast(m1 - t1) : 1.0f;
                    m0 = up0 ? t0 : m0;
                    m1 = up1 ? t1 : m1;
                    l0 *= d0;
                    l1 *= d1;
                    if (t > w.t0) {
                        const int pt = tile - 1;
                        ok = mbar_wait(smem_addr(&s.kv_empty[pt % stages]), (pt / stages) & 1, status);
                        ok = __all_sync(~0u, ok);
                        if (!ok)
                            break;
                        tc_fence_after();
                        for (int n = 0; n < p.v_dim; n += 32) {
                            float o[16];
                            tmem_ld_16x256(my_lanes + n, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                o[i] *= (i & 2) ? d1 : d0;
                            tmem_st_16x256(my_lanes + n, o);
                        }
                        tmem_wait_st();
                    }
                }
                const float ref0 = m0 == -INFINITY ? 0.0f : m0, ref1 = m1 == -INFINITY ? 0.0f : m1;
                uint32_t pk[8];  // of x[2 i], x[2 i + 1]
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float ref = (i & 1) ? ref1 : ref0;
                    float a = exp2_fast(x[2 * i] - ref), e = exp2_fast(x[2 * i + 1] - ref);
                    if (i & 1)
                        l1 += a + e;
                    else
                        l0 += a + e;
                    if constexpr (BITS8) {
                        // a hidden row's scale may be anything: its weight stays 0
                        a = a == 0.0f ? 0.0f : a * rs[i / 2].x;
                        e = e == 0.0f ? 0.0f : e * rs[i / 2].y;
                    }
                    pk[i] = f2_to_bf16x2(make_float2(a, e));
                }
                if (tile >= 2) {
                    // the buffer's last reader
                    const int pt = tile - 2;
                    ok = mbar_wait(smem_addr(&s.kv_empty[pt % stages]), (pt / stages) & 1, status);
                    ok = __all_sync(~0u, ok);
                    if (!ok)
                        break;
                }
#pragma unroll
                for (int g8 = 0; g8 < 4; ++g8) {
                    uint8_t *at = p_mem + r0 * 128 + (((4 * b + g8) ^ (r0 & 7)) << 4) + 2 * cq;
                    *reinterpret_cast<uint32_t *>(at) = pk[2 * g8];
                    *reinterpret_cast<uint32_t *>(at + 8 * 128) = pk[2 * g8 + 1];
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&s.p_full[b]));
            }
            if (!ok)
                break;
            // ---- output: whole items are finished here, parts go to the workspace
            const bool done = w.t0 == 0 && w.t1 == w.nt;
            if (w.t1 > w.t0) {
                const int pt = tile - 1;
                ok = mbar_wait(smem_addr(&s.kv_empty[pt % stages]), (pt / stages) & 1, status);
                ok = __all_sync(~0u, ok);
                if (!ok)
                    break;
                tc_fence_after();
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                l0 += __shfl_xor_sync(~0u, l0, o);
                l1 += __shfl_xor_sync(~0u, l1, o);
            }
            // O is read a row a thread, by threads 0-15
            const int row = warp * 16 + (lane & 15), from_lane = 4 * (lane & 7);
            const float ma = __shfl_sync(~0u, m0, from_lane), mb = __shfl_sync(~0u, m1, from_lane);
            const float la = __shfl_sync(~0u, l0, from_lane), lb = __shfl_sync(~0u, l1, from_lane);
            const float m = lane & 8 ? mb : ma, l = lane & 8 ? lb : la;
            const bool live = row < item_rows, write = live && lane < 16;
            if (done) {
                const int head = live ? (w.item() * kTile + row) % p.n_heads : 0;
                const float sink = p.sink ? __ldg(p.sink + head) * kLog2E : -INFINITY;
                const float top = fmaxf(m, sink), ref = top == -INFINITY ? 0.0f : top;
                const float down = exp2_fast(m - ref), tot = l * down + exp2_fast(sink - ref);
                const float inv = tot == 0.0f ? 0.0f : down / tot;
                if (write && p.lse)
                    p.lse[out_row + row] = tot == 0.0f ? -INFINITY : (ref + log2f(tot)) * kLn2;
                uint8_t *dst = static_cast<uint8_t *>(p.out) + (out_row + row) * p.v_dim * 2;
                for (int n = 0; n < p.v_dim; n += 32) {
                    float o[32];
                    if (w.t1 > w.t0) {
                        tmem_ld_32x32(my_lanes + n, o);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = 0.0f;
                    }
                    if (write)
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            *reinterpret_cast<uint4 *>(dst + (n + i) * 2) = make_uint4(
                                f2_to_bf16x2(make_float2(o[i] * inv, o[i + 1] * inv)),
                                f2_to_bf16x2(make_float2(o[i + 2] * inv, o[i + 3] * inv)),
                                f2_to_bf16x2(make_float2(o[i + 4] * inv, o[i + 5] * inv)),
                                f2_to_bf16x2(make_float2(o[i + 6] * inv, o[i + 7] * inv)));
                }
            } else {
                const int64_t slot = 2 * (int64_t)c + (w.t0 == 0 ? 1 : 0);
                if (write)
                    plan.part_ml[slot * kTile + row] = make_float2(m, l);
                float *dst = plan.part_o + (slot * kTile + row) * p.v_dim;
                for (int n = 0; n < p.v_dim; n += 32) {
                    float o[32];
                    tmem_ld_32x32(my_lanes + n, o);
                    tmem_wait_ld();
                    if (write)
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<float4 *>(dst + n + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                }
                if (w.t0 == 0 && tid == 0) {
                    // the item's last unit is the block's last so far plus the tiles it has not taken
                    const long long last = unit - 1 + (w.nt - w.t1);
                    plan.joins[c] = make_int4((int)out_row, item_rows, (int)(((last + 1) * g - 1) / total), 1);
                }
            }
            tc_fence_before();
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------ matrix products
        // The warp stays together and one thread of it issues: the operands of tcgen05.mma are warp-uniform registers,
        // and a single thread running the loop alone would have each of them moved there, at some 100 cycles an MMA.
        const uint32_t tm = __shfl_sync(~0u, tmem, 0);
        const uint64_t q_desc = mma_operand(smem_addr(q_mem), 16, 1024), k_desc = mma_operand(smem_addr(kv_mem), 16, 1024);
        const uint64_t p_desc = mma_operand(smem_addr(p_mem), 16, 1024);
        const uint64_t v_desc = mma_operand(smem_addr(kv_mem), kChunk, 1024);
        constexpr uint32_t kStep = kChunk >> 4, kQueryStep = kQueryChunk >> 4;  // of a descriptor's address
        const uint32_t shape_s = mma_shape(kTile, kRows, false);
        const int stages_u = __shfl_sync(~0u, stages, 0), nk_u = __shfl_sync(~0u, nk, 0);
        auto product = [&](int tile, int st, bool first) {  // O (+)= P V
            ok = mbar_wait(smem_addr(&s.p_full[tile & 1]), (tile >> 1) & 1, status);
            ok = __all_sync(~0u, ok);
            if (!ok)
                return;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t v = v_desc + (uint32_t)(st * nk_u) * kStep;
                const uint64_t pa = p_desc + (tile & 1) * 4;
                for (int n = 0; n < p.v_dim; n += 256) {
                    const uint32_t shape = mma_shape(kTile, min(256, p.v_dim - n), true);
#pragma unroll
                    for (int k = 0; k < kRows / 16; ++k)
                        mma_bf16(tm + n, pa + k * 2, v + (n / 64) * kStep + k * 128, shape, !first || k > 0);
                }
                mma_commit(smem_addr(&s.kv_empty[st]));
            }
            __syncwarp();
        };
        int tile = 0, segment = 0, st = 0, phase = 0;
        Walk w(p, s, units);
        while (ok && __shfl_sync(~0u, (int)w.next(), 0)) {
            const int t0 = __shfl_sync(~0u, w.t0, 0), t1 = __shfl_sync(~0u, w.t1, 0);
            if (t1 <= t0)
                continue;
            ok = mbar_wait(smem_addr(&s.q_full), segment++ & 1, status);
            ok = __all_sync(~0u, ok);
            int before = 0;
            for (int t = t0; t < t1 && ok; ++t, ++tile) {
                const int b = tile & 1;
                ok = mbar_wait(smem_addr(&s.kv_full[st]), phase, status);
                ok = __all_sync(~0u, ok);
                if (!ok)
                    break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t k = k_desc + (uint32_t)(st * nk_u) * kStep;
                    const uint32_t d = tm + (16u << 16) + b * kRows;
                    for (int ch = 0; ch < nk_u; ++ch)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_bf16(d, q_desc + ch * kQueryStep + i * 2, k + ch * kStep + i * 2, shape_s, ch > 0 || i > 0);
                    mma_commit(smem_addr(&s.s_full[b]));
                    if (t + 1 == t1)
                        mma_commit(smem_addr(&s.q_empty));
                }
                __syncwarp();
                if (t > t0)
                    product(tile - 1, before, t - 1 == t0);
                before = st;
                if (++st == stages_u) {
                    st = 0;
                    phase ^= 1;
                }
            }
            if (ok)
                product(tile - 1, before, t1 - 1 == t0);
        }
        // nothing may be in flight when the block frees its memory, a wait that gave up included
        if (elect_one())
            mma_commit(smem_addr(&s.drained));
        __syncwarp();
        mbar_wait(smem_addr(&s.drained), 0, status);
        __syncwarp();
    } else if (BITS8 || warp != kTmaWarp) {
        // ------------------------------------------------ queries, and 8-bit rows, through registers
        const int lw = warp - (BITS8 ? kMmaWarp : kTmaWarp) - 1;
        const uint8_t *cache = static_cast<const uint8_t *>(p.cache);
        int tile = 0, segment = 0;
        Walk w(p, s, units);
        while (ok && w.next()) {
            if (w.t1 <= w.t0)
                continue;
            const int item_rows = min(kTile, w.q.nq * p.n_heads - w.item() * kTile);
            {
                // 64 rows, four a warp at a time; the products S of the segment before have to be done
                constexpr int kTurns = kTile / (4 * kQueryArrivals);
                uint4 v[kTurns][NKB];
#pragma unroll
                for (int i = 0; i < kTurns; ++i) {
                    const int row = (i * kQueryArrivals + lw) * 4 + (lane >> 3), flat = w.item() * kTile + row;
                    const uint8_t *src = static_cast<const uint8_t *>(p.q) + (lane & 7) * 16;
                    if (row < item_rows)
                        src += ((int64_t)(w.q.first + flat / p.n_heads) * p.q_token_stride +
                                (int64_t)(flat % p.n_heads) * p.q_head_stride) * 2;
#pragma unroll
                    for (int ch = 0; ch < NKB; ++ch)
                        v[i][ch] = ch < nk && row < item_rows ? __ldg(reinterpret_cast<const uint4 *>(src + ch * 128)) : zero4();
                }
                if (segment > 0) {
                    ok = mbar_wait(smem_addr(&s.q_empty), (segment - 1) & 1, status);
                    ok = __all_sync(~0u, ok);
                    if (!ok)
                        break;
                }
                ++segment;
#pragma unroll
                for (int i = 0; i < kTurns; ++i) {
                    const int row = (i * kQueryArrivals + lw) * 4 + (lane >> 3);
                    uint8_t *dst = q_mem + row * 128 + (((lane & 7) ^ (row & 7)) << 4);
#pragma unroll
                    for (int ch = 0; ch < NKB; ++ch)
                        if (ch < nk)
                            *reinterpret_cast<uint4 *>(dst + ch * kQueryChunk) = v[i][ch];
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&s.q_full));
            }
            if constexpr (BITS8) {
                const int end = visible(p, w.q, last_token(p, w.q, w.item()));
                const int32_t *table = p.block_table + (int64_t)w.r * p.table_stride;
                for (int t = w.t0; t < w.t1; ++t, ++tile) {
                    const int st = tile % stages;
                    // the warp's rows 4 lw ... 4 lw + 3 of the tile: lane % 4 looks one up
                    const int j = t * kRows + lw * 4 + (lane & 3);
                    int64_t slot = -1;
                    if (j < end) {
                        const int page = __ldg(table + j / p.page_size);
                        if (page >= 0 && page < p.n_pages)
                            slot = (int64_t)page * p.page_size + j % p.page_size;
                    }
                    const uint32_t valid = __ballot_sync(~0u, slot >= 0) & 0xfu;
                    // a lane brings 16 columns of every second chunk
                    const int row = lane >> 3, odd = lane >> 2 & 1, quarter = lane & 3;
                    const int64_t at = __shfl_sync(~0u, slot, row);
                    constexpr int kHalf = (NKB + 1) / 2;
                    uint4 v[kHalf];
                    const uint8_t *src = cache + at * p.cache_stride + odd * 64 + quarter * 16;
#pragma unroll
                    for (int i = 0; i < kHalf; ++i)
                        v[i] = 2 * i + odd < nk && at >= 0 ? __ldg(reinterpret_cast<const uint4 *>(src + i * 128)) : zero4();
                    const float sc = slot >= 0 ? __ldg(p.row_scales + slot) : 0.0f;
                    if (tile >= stages) {
                        ok = mbar_wait(smem_addr(&s.kv_empty[st]), (tile / stages - 1) & 1, status);
                        ok = __all_sync(~0u, ok);
                        if (!ok)
                            break;
                    }
                    if (lane < 4)
                        s.scales[st][lw * 4 + lane] = sc;
                    const int r = lw * 4 + row;
                    uint8_t *dst = kv_mem + (st * nk + odd) * kChunk + r * 128;
#pragma unroll
                    for (int i = 0; i < kHalf; ++i)
                        if (2 * i + odd < nk)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const uint32_t a = u ? v[i].z : v[i].x, e = u ? v[i].w : v[i].y;
                                *reinterpret_cast<uint4 *>(dst + 2 * i * kChunk + (((2 * quarter + u) ^ (r & 7)) << 4)) =
                                    make_uint4(bf16x2_of_e4m3x2(a & 0xffffu), bf16x2_of_e4m3x2(a >> 16),
                                               bf16x2_of_e4m3x2(e & 0xffffu), bf16x2_of_e4m3x2(e >> 16));
                            }
                    if (lane == 0)
                        s.valid[st][lw] = (uint8_t)valid;
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_addr(&s.kv_full[st]));
                }
            }
        }
    } else if constexpr (!BITS8) {
        // ------------------------------------------------ bf16 rows by TMA
        const uint32_t kv_smem = smem_addr(kv_mem);
        const int none = (int)(p.n_pages * p.page_size);  // a row past the end reads as zeros
        int tile = 0;
        Walk w(p, s, units);
        while (ok && w.next()) {
            const int end = visible(p, w.q, last_token(p, w.q, w.item()));
            const int32_t *table = p.block_table + (int64_t)w.r * p.table_stride;
            for (int t = w.t0; t < w.t1; ++t, ++tile) {
                const int st = tile % stages;
                auto look_up = [&](int j) {
                    if (j < end) {
                        const int page = __ldg(table + j / p.page_size);
                        if (page >= 0 && page < p.n_pages)
                            return page * p.page_size + j % p.page_size;
                    }
                    return none;
                };
                const int slot = look_up(t * kRows + lane);
                const uint32_t valid = __ballot_sync(~0u, slot != none);
                if (tile >= stages) {
                    ok = mbar_wait(smem_addr(&s.kv_empty[st]), (tile / stages - 1) & 1, status);
                    ok = __all_sync(~0u, ok);
                    if (!ok)
                        break;
                }
                const uint32_t bar = smem_addr(&s.kv_full[st]), dst = kv_smem + st * nk * kChunk;
                if (lane == 0) {
                    *reinterpret_cast<uint32_t *>(s.valid[st]) = valid;
                    mbar_arrive_expect_tx(bar, nk * kChunk);
                }
                __syncwarp();
                if (plan.box_rows > 0 && valid == ~0u) {
                    const int runs = kRows / plan.box_rows;
                    for (int i = lane; i < ((runs * nk + 31) & ~31); i += 32) {
                        const int ch = i / runs, row = i % runs * plan.box_rows;
                        const int r = __shfl_sync(~0u, slot, row);
                        if (ch < nk)
                            tma_load_2d(dst + ch * kChunk + row * 128, &boxes, ch * 64, r, bar);
                    }
                } else {
                    const int four = lane & 7;  // rows 4 four ... 4 four + 3, every fourth chunk
                    int r[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        r[k] = __shfl_sync(~0u, slot, four * 4 + k);
                    for (int ch = lane >> 3; ch < nk; ch += 4)
                        tma_gather4(dst + ch * kChunk + four * 512, &single, ch * 64, r[0], r[1], r[2], r[3], bar);
                }
            }
        }
        // no copy outlives the block, after a wait that gave up either
        if (lane == 0)
            for (int k = max(0, tile - stages); k < tile; ++k)
                mbar_wait(smem_addr(&s.kv_full[k % stages]), (k / stages) & 1, status);
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_free(tmem, plan.tmem_columns);
    }
}

// Joins the parts of the items that cross block boundaries: block (c, y) takes four rows of the item whose first part
// block c of the kernel above wrote (its slot 1), with the slots 0 of the blocks after it up to the item's last.
__global__ void __launch_bounds__(512) latent_join_kernel(const AttnParams p, const MmaPlan plan)
{
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x;
    const int4 j = plan.joins[c];
    const int row = blockIdx.y * 4 + threadIdx.y;
    if (!j.w || row >= j.y)
        return;
    const int64_t out_row = (int64_t)j.x + row;
    const int head = (int)(out_row % p.n_heads);
    const float sink = p.sink ? __ldg(p.sink + head) * kLog2E : -INFINITY;
    auto part = [&](int k) { return (k == c ? 2 * (int64_t)c + 1 : 2 * (int64_t)k) * kTile + row; };
    float top = sink;
    for (int k = c; k <= j.z; ++k)
        top = fmaxf(top, plan.part_ml[part(k)].x);
    const float ref = top == -INFINITY ? 0.0f : top;
    float tot = exp2_fast(sink - ref);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    const int col = threadIdx.x * 4;
    for (int k = c; k <= j.z; ++k) {
        const int64_t at = part(k);
        const float2 ml = plan.part_ml[at];
        const float w = exp2_fast(ml.x - ref);
        tot = fmaf(w, ml.y, tot);
        if (col < p.v_dim) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(plan.part_o + at * p.v_dim + col));
            o.x = fmaf(w, v.x, o.x);
            o.y = fmaf(w, v.y, o.y);
            o.z = fmaf(w, v.z, o.z);
            o.w = fmaf(w, v.w, o.w);
        }
    }
    const float inv = tot == 0.0f ? 0.0f : 1.0f / tot;
    if (col < p.v_dim)
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + out_row * p.v_dim + col) =
            make_uint2(f2_to_bf16x2(make_float2(o.x * inv, o.y * inv)), f2_to_bf16x2(make_float2(o.z * inv, o.w * inv)));
    if (p.lse && threadIdx.x == 0)
        p.lse[out_row] = tot == 0.0f ? -INFINITY : (ref + log2f(tot)) * kLn2;
}

template <bool BITS8, int NKB>
cudaError_t go(const AttnParams &p, const MmaPlan &plan, unsigned *status, cudaStream_t st)
{
    auto kern = latent_mma_kernel<BITS8, NKB>;
    cudaError_t e = allow_max_smem(reinterpret_cast<const void *>(kern));
    CUtensorMap boxes = {}, single = {};
    if (!BITS8 && e == cudaSuccess && p.n_pages > 0 && p.width > 0) {
        const int64_t rows = p.n_pages * p.page_size;
        e = make_tensor_map_rows(&single, p.cache, rows, p.head_dim, p.cache_stride, 1);
        if (e == cudaSuccess && plan.box_rows > 0)
            e = make_tensor_map_rows(&boxes, p.cache, rows, p.head_dim, p.cache_stride, plan.box_rows);
    }
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = st;
    cfg.gridDim = dim3(plan.blocks);
    cfg.blockDim = dim3(kThreadsOf<BITS8>);
    cfg.dynamicSmemBytes = plan.smem;
    e = cudaLaunchKernelEx(&cfg, kern, p, plan, boxes, single, status);
    if (e != cudaSuccess)
        return e;
    cfg.gridDim = dim3(plan.blocks, kTile / 4);
    cfg.blockDim = dim3((p.v_dim + 3) / 4, 4);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, latent_join_kernel, p, plan);
}

MmaPlan make_plan(const AttnParams &p, int num_sms)
{
    constexpr size_t kLimit = 227 * 1024 - sizeof(Shared);
    MmaPlan m{};
    m.nk = p.head_dim / 64;
    const size_t fixed = (size_t)(m.nk + 1) * kQueryChunk + 1024;  // queries, P, alignment
    m.stages = (int)((kLimit - fixed) / ((size_t)m.nk * kChunk));
    m.stages = m.stages > kMaxStages ? kMaxStages : m.stages;
    m.smem = fixed + (size_t)m.stages * m.nk * kChunk;
    for (m.box_rows = kRows; p.page_size % m.box_rows; m.box_rows /= 2) {}
    m.box_rows = m.box_rows < 8 ? 0 : m.box_rows;  // eight rows are the swizzle's period
    // more than half an SM's shared memory: one block an SM (it owns the tensor memory), and room for the offsets of
    // kMaxRequests requests
    m.smem = m.smem < 120 * 1024 ? 120 * 1024 : m.smem;
    m.tmem_columns = p.v_dim > 256 ? 512 : p.v_dim > 128 ? 256 : 128;
    m.blocks = num_sms;
    m.min_units = 8;
    return m;
}

}  // namespace

bool latent_mma_supported(const AttnParams &p)
{
    return p.head_dim % 64 == 0 && p.head_dim <= 576 && p.v_dim % 64 == 0 && p.v_dim <= 512;
}

size_t latent_mma_workspace(const AttnParams &p, int num_sms)
{
    const MmaPlan m = make_plan(p, num_sms);
    return (size_t)m.blocks * (2 * kTile * ((size_t)p.v_dim * sizeof(float) + sizeof(float2)) + sizeof(int4));
}

cudaError_t launch_latent_mma(const AttnParams &p, void *workspace, int num_sms, unsigned *status, cudaStream_t st)
{
    MmaPlan m = make_plan(p, num_sms);
    m.part_o = static_cast<float *>(workspace);
    m.part_ml = reinterpret_cast<float2 *>(m.part_o + (size_t)m.blocks * 2 * kTile * p.v_dim);
    m.joins = reinterpret_cast<int4 *>(m.part_ml + (size_t)m.blocks * 2 * kTile);
    const bool bits8 = p.cache_dtype == CSA_DTYPE_E4M3;
    if (m.nk <= 4)
        return bits8 ? go<true, 4>(p, m, status, st) : go<false, 4>(p, m, status, st);
    return bits8 ? go<true, 9>(p, m, status, st) : go<false, 9>(p, m, status, st);
}

}  // namespace csa
