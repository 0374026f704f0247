// Attention over a paged cache of shared latent rows on the tensor cores (tcgen05).
//
// The query rows of a request are its (token, head) pairs, in order; all of them read the same cache rows.  An item is
// 64 such rows.  For each tile of R = 48 or 64 cache rows:
//
//   S = Q K^T          64 x R, K = head_dim: both operands K-major in shared memory
//   P = exp2(S f - m)  f = scale log2 e, m the row's reference; l += sum P; P to bf16 in shared memory
//   O = O + P V        64 x v_dim, K = R cache rows; V is the K tile itself, read with its rows along K
//
// so a cache row is fetched once and used for both products.  m is raised (O and l scaled down) only when a logit
// exceeds it by 2^8: P stays below 2^8, which bf16 and the fp32 sums hold as well as values below one, and O is
// rarely touched outside the tensor core.
//
// Tensor memory: a 64-row accumulator takes 16 of each 32 lanes, so O (up to 512 columns) has the lower sixteen and
// four S tiles the upper sixteen.  64 query rows, not 128: O of 128 x 512 alone would fill tensor memory, and K tiles
// of 576 columns and 128 query rows would not fit shared memory twice.
//
// Shared memory: a tile lies in groups of eight rows, a group chunk by chunk (64 columns), a chunk as eight swizzled rows
// of 128 bytes, so that one TMA copy brings any run of whole groups with all their columns: the issue of a copy costs
// some 80 cycles, and a copy a chunk bounded the kernel.
//
// Warps: 0-3 exponentials and output (each owns 16 query rows: its quarter of the lanes), 4 issues the MMAs.  Pages of
// whole groups of bf16 rows: warp 5 issues TMA copies, warps 6-9 bring the next item's queries through registers.
// Other pages, and 8-bit rows: warps 5 and on take turns at the groups, bring them to registers, widen 8-bit values to
// bf16 (exact) and write the swizzled layout.  An 8-bit row's scale multiplies S by column and P before its rounding,
// so it costs no precision.
//
// Work is cut evenly: an item counts three units for its queries and output and one for each tile; block c takes the units
// [c T / G, (c+1) T / G) of the T units.  Items that cross a cut leave (O, m, l) of their parts in the workspace and a
// second kernel joins them in order.  Nothing else depends on the grid, and no order on timing.
//
// SHARED: a request's first rows may be dealt with apart, as a prefix that it shares (csa_shared.cu).  Its rows here are those
// behind; every item leaves its parts, which csa_shared.cu joins with the prefix's.
#include <cuda.h>
#include <cuda_fp8.h>

#include "csa_launch.h"
#include "csa_serving_launch.h"
#include "csa_shared.cuh"
#include "csa_tcgen05.cuh"

namespace csa {
namespace {

enum Rows { kTma, kRegisters, kBits8 };           // how rows come: TMA copies, through registers, 8 bits through registers

constexpr int kTile = 64;                         // query rows of an item
constexpr int kQueryChunk = kTile * 128;          // bytes of 64 columns of an item's queries
constexpr int kGroupChunk = 8 * 128;              // bytes of 64 columns of eight rows
constexpr int kSoftWarps = 4;
constexpr int kMmaWarp = 4;
// Blocks an SM: two where the shared memory and tensor memory of each allow it (rows of up to 256 columns), whose waits
// then overlap (64 heads: 1024 tokens over 4096 rows of 128 columns 377 us with one, 240 with two, a decode step of 64 requests
// of up to 8192 rows 42.4 and 36.3; of 256 columns 383 and 332, but the decode step 46.6 and 52.5).  Rows through registers
// are brought by eight warps or, to leave registers for two blocks, four, which then spill some 250 bytes a thread (decode
// steps of 64 and 128 8-bit columns 48.7 and 53.3 us with one block, 42.9 and 49.3 with two); for their 256 columns one
// block is better (55.7 and 63.1 us, in pages of 50 bf16 rows 66 and 75).
constexpr int per_sm(Rows how, int nk) { return nk <= (how == kTma ? 4 : 3) ? 2 : 1; }
constexpr int load_warps(Rows how, int nk) { return 8 / per_sm(how, nk); }
constexpr int kTmaWarp = 5;                       // rows by TMA
constexpr int kQueryWarps = 4;                    // rows by TMA: warps that bring queries
template <Rows ROWS, int NK>
constexpr int kThreadsOf = 32 * (ROWS == kTma ? kTmaWarp + 1 + kQueryWarps : kMmaWarp + 1 + load_warps(ROWS, NK));
constexpr int kMaxStages = 4;
constexpr int kKept = 2048;                       // requests whose facts are kept in shared memory while work is cut
constexpr int kScores = 4;                        // S tiles in tensor memory
constexpr float kLog2E = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kRaise = 8.0f;                    // log2 of how far a logit may exceed the reference

struct MmaPlan {
    int stages;
    int blocks;       // G
    bool helpers;     // the join: blocks for every part, not for the first of an item alone
    int p_buffers;    // 1 or 2
    int box_groups;   // groups of eight rows of the larger TMA copy
    uint32_t tmem_columns;
    size_t smem;
    float *part_o;    // [2 blocks][64][v_dim]
    float2 *part_ml;  // [2 blocks][64]  (m, l)
    int4 *joins;      // [2 blocks]  of each part: query row, rows (0: no part), the item's first and last block
};

struct Shared {
    uint64_t kv_full[kMaxStages], kv_empty[kMaxStages], s_full[kScores], p_full[2], q_full, q_empty, flags, drained;
    long long sums[16];
    long long total;
    int r, m, off, index;        // where the block's units begin; the item's number in all
    int first[4];                // and the facts of request r
    uint32_t tmem;
    alignas(16) float scales[kMaxStages][64];
    alignas(8) uint8_t missing[kMaxStages][8];  // bit i % 8 of byte i / 8: row i of the tile lies in no page of the cache
    alignas(8) uint16_t poison[2][kSoftWarps];
};

// What an item is made of.
struct Request {
    int first;    // first token
    int nq;
    int before;   // tokens of the request before its first new one (may be negative)
    int items;
};

struct NoPrefix {};
template <bool SHARED> struct PrefixOf {
    using type = NoPrefix;
};
template <> struct PrefixOf<true> {
    using type = SharedPlan;
};
template <bool SHARED> using Prefix = typename PrefixOf<SHARED>::type;

// The rows of request r that its group's prefix part has (whole pages), and the group.
__device__ __forceinline__ int2 own_of(const NoPrefix &, int) { return make_int2(0, -1); }
__device__ __forceinline__ int2 own_of(const SharedPlan &s, int r) { return __ldcg(s.own + r); }

template <bool SHARED> __device__ __forceinline__ Request request(const AttnParams &p, const Prefix<SHARED> &prefix, int r)
{
    Request q;
    q.first = max(__ldg(p.cu_q + r), 0);
    const int64_t end = min((int64_t)__ldg(p.cu_q + r + 1), p.n_tokens);
    q.nq = (int)max(end - q.first, (int64_t)0);
    q.before = __ldg(p.seq_lens + r) - (__ldg(p.cu_q + r + 1) - q.first);
    q.items = (int)(((int64_t)q.nq * p.n_heads + kTile - 1) / kTile);
    if constexpr (SHARED)
        q.before -= own_of(prefix, r).x * p.ratio;  // (the prefix part has no more rows than every new token sees)
    return q;
}

__device__ __forceinline__ int visible(const AttnParams &p, const Request &q, int token)
{
    const int held = q.before + token + 1;
    return held <= 0 ? 0 : min((int)p.by_ratio.quotient((uint32_t)held), p.width * p.page_size);
}

// (all in 32 bits and by multiplication: the tokens times the heads stay below 2^31, and divisions, 64-bit ones above
// all, made half of a block's first 7000 cycles)
__device__ __forceinline__ int last_token(const AttnParams &p, const Request &q, int m)
{
    return (int)p.by_heads.quotient(min((uint32_t)(m + 1) * kTile, (uint32_t)q.nq * (uint32_t)p.n_heads) - 1);
}

template <int R> __device__ __forceinline__ int item_tiles(const AttnParams &p, const Request &q, int m)
{
    return (visible(p, q, last_token(p, q, m)) + R - 1) / R;
}

// The block's segments, walked alike by every role.
template <bool SHARED, int R> struct Walk {
    const AttnParams &p;
    const Prefix<SHARED> &prefix;
    Request q;
    int r, m, off;
    long long left;
    int nt, t0, t1, index;
    __device__ Walk(const AttnParams &p_, const Prefix<SHARED> &prefix_, const Shared &s, long long units)
        : p(p_), prefix(prefix_), q{s.first[0], s.first[1], s.first[2], s.first[3]}, r(s.r), m(s.m), off(s.off), left(units), index(s.index - 1)
    {
    }
    // the next segment: tiles [t0, t1) of item (r, m); nt == 0 (t0 == t1) is an item that sees nothing
    __device__ bool next()
    {
        while (left > 0) {
            while (m >= q.items) {
                if (++r >= p.n_req)
                    return false;
                m = 0;
                q = request<SHARED>(p, prefix, r);
            }
            nt = item_tiles<R>(p, q, m);
            const Segment s = segment_of(nt, off, left);
            t0 = s.t0;
            t1 = s.t1;
            left -= s.take;
            off = 0;
            ++m;
            ++index;
            if (s.some)
                return true;
        }
        return false;
    }
    __device__ int item() const { return m - 1; }
    // The request's pages behind its prefix.
    __device__ const int32_t *table() const
    {
        const int32_t *t = p.block_table + (int64_t)r * p.table_stride;
        if constexpr (SHARED)
            t += p.by_page.quotient((uint32_t)own_of(prefix, r).x);
        return t;
    }
};

__device__ __forceinline__ uint4 zero4() { return make_uint4(0, 0, 0, 0); }

// Read-only loads that stay where they are written: ahead of the waits that they are to overlap.
__device__ __forceinline__ uint4 load_now(const uint8_t *at)
{
    uint4 v;
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(at));
    return v;
}

__device__ __forceinline__ int load_now(const int32_t *at)
{
    int v;
    asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(v) : "l"(at));
    return v;
}

__device__ __forceinline__ bool nonfinite_bf16(uint32_t w)
{
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

__device__ __forceinline__ uint32_t bf16x2_of_e4m3x2(uint32_t two)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    return f2_to_bf16x2(__half22float2(*reinterpret_cast<const __half2 *>(&h)));
}

template <bool SHARED, Rows ROWS, int NK, int R>
__global__ void __launch_bounds__(kThreadsOf<ROWS, NK>, per_sm(ROWS, NK))
latent_mma_kernel(const AttnParams p, const MmaPlan plan, const Prefix<SHARED> prefix, const __grid_constant__ CUtensorMap boxes,
                  const __grid_constant__ CUtensorMap groups, unsigned *status)
{
    constexpr int kThreads = kThreadsOf<ROWS, NK>;
    constexpr int kLoadWarps = load_warps(ROWS, NK);
    constexpr int kQueryArrivals = ROWS == kTma ? kQueryWarps : kLoadWarps;
    constexpr int kGroups = R / 8;
    constexpr int kGroupBytes = NK * kGroupChunk, kTileBytes = kGroups * kGroupBytes;
    extern __shared__ uint8_t raw[];
    __shared__ Shared s;
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const int stages = plan.stages;
    uint8_t *q_mem = base, *p_mem = q_mem + NK * kQueryChunk, *kv_mem = p_mem + plan.p_buffers * kQueryChunk;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(smem_addr(&s.kv_full[i]), ROWS == kTma ? 1 : kGroups);
            mbar_init(smem_addr(&s.kv_empty[i]), 1);
            *reinterpret_cast<uint64_t *>(s.missing[i]) = 0;
        }
        for (int i = 0; i < kScores; ++i)
            mbar_init(smem_addr(&s.s_full[i]), 1);
        // (two, by the tile's parity: a warp may be a tile ahead of another)
        mbar_init(smem_addr(&s.p_full[0]), kSoftWarps);
        mbar_init(smem_addr(&s.p_full[1]), kSoftWarps);
        mbar_init(smem_addr(&s.q_full), kQueryArrivals);
        mbar_init(smem_addr(&s.q_empty), 1);
        mbar_init(smem_addr(&s.flags), kSoftWarps);
        mbar_init(smem_addr(&s.drained), 1);
        mbar_init_fence();
    }
    // SHARED: what this kernel reads was there before the one in front of it (the prefixes') let this one begin, so its blocks
    // begin as that one's end, and wait for its end at their own.
    if constexpr (!SHARED)
        pdl_wait();
    pdl_trigger();
    if (warp == kMmaWarp)
        tmem_alloc(smem_addr(&s.tmem), plan.tmem_columns);

    // ---- where this block's units begin: prefix sums of items over requests (in the space of the tiles), then of
    // units over equal stretches of items, a stretch a thread
    int *items = reinterpret_cast<int *>(base);
    Request *kept = reinterpret_cast<Request *>(base + ((kMaxRequests + 4) & ~3) * sizeof(int));
    auto fact = [&](int r) { return r < kKept ? kept[r] : request<SHARED>(p, prefix, r); };
    {
        int run = 0;
        int *warp_sum = reinterpret_cast<int *>(s.sums);
        for (int at = 0; at < p.n_req; at += kThreads) {
            const int r = at + tid;
            int n = 0;
            if (r < p.n_req) {
                const Request q = request<SHARED>(p, prefix, r);
                n = q.items;
                if (r < kKept)
                    kept[r] = q;
            }
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
        // Two passes of one loop (its instructions are fetched once): a thread's units, then, with the sums before it
        // known, which item the block's first unit lies in.
        long long mine = 0, first = 0, total = 0, from = 0;
        bool here = true;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
            if (lo < hi && here) {
                int r = 0;  // items[r] <= lo < items[r + 1]
                for (int top = p.n_req; top - r > 1;) {
                    const int mid = (r + top) >> 1;
                    if (items[mid] <= lo)
                        r = mid;
                    else
                        top = mid;
                }
                Request q = fact(r);
                int m = lo - items[r];
                long long at = first;
                for (int i = lo; i < hi; ++i, ++m) {
                    while (m >= q.items) {
                        q = fact(++r);
                        m = 0;
                    }
                    const int units = item_tiles<R>(p, q, m) + kHead;
                    if (pass == 1 && from >= at && from < at + units) {
                        s.r = r;
                        s.m = m;
                        s.off = (int)(from - at);
                        s.index = i;
                        s.first[0] = q.first;
                        s.first[1] = q.nq;
                        s.first[2] = q.before;
                        s.first[3] = q.items;
                    }
                    at += units;
                }
                mine = at - first;
            }
            if (pass == 0) {
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
                long long before = 0;
                for (int i = 0; i < kThreads / 32; ++i) {
                    before += i < warp ? s.sums[i] : 0;
                    total += s.sums[i];
                }
                first = before + a - mine;
                const int g = sharing(total, plan.blocks);
                from = cut(total, blockIdx.x, g);
                here = blockIdx.x < g && from >= first && from < first + mine;
            }
        }
        if (tid == 0) {
            s.total = total;
            if constexpr (SHARED)
                if (blockIdx.x == 0)
                    *prefix.n_items = min(run, prefix.max_own);
        }
    }
    // TMA copies and the tensor core take over the space that these sums were in
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const long long total = s.total;
    const int g = sharing(total, plan.blocks), c = blockIdx.x;
    const long long from = cut(total, c, g), units = c < g ? cut(total, c + 1, g) - from : 0;
    const uint32_t tmem = s.tmem;
    bool ok = true;

    if (warp < kSoftWarps) {
        // ------------------------------------------------ exponentials and output
        if (!SHARED && tid == 0)
            plan.joins[2 * c] = plan.joins[2 * c + 1] = make_int4(0, 0, 0, 0);
        const uint32_t my_lanes = tmem + ((uint32_t)(warp * 32) << 16);
        // S: this thread has columns 8 g + 2 (lane % 4) + {0, 1} of rows r0 (x[4g], x[4g + 1]) and r0 + 8
        const int r0 = warp * 16 + lane / 4, cq = 2 * (lane & 3);
        const float f = p.scale * kLog2E;
        int tile = 0;                             // tiles of the block so far
        int flagged = 0;                          // of them, those whose rows were looked through
        long long unit = from;
        Walk<SHARED, R> w(p, prefix, s, units);
        while (ok) {
            const long long left = w.left;
            if (!w.next())
                break;
            unit += left - w.left;  // one past the segment's last unit
            const int item_rows = min(kTile, w.q.nq * p.n_heads - w.item() * kTile);
            const int64_t out_row = (int64_t)w.q.first * p.n_heads + (int64_t)w.item() * kTile;
            auto seen_by = [&](int row) {
                return row < item_rows ? visible(p, w.q, (int)p.by_heads.quotient(w.item() * kTile + row)) : 0;
            };
            const int seen0 = seen_by(r0), seen1 = seen_by(r0 + 8);
            const int all_see = visible(p, w.q, (int)p.by_heads.quotient((uint32_t)w.item() * kTile));
            const int end = visible(p, w.q, last_token(p, w.q, w.item()));
            const bool whole = item_rows == kTile;
            float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;  // l: this thread's columns only
            for (int t = w.t0; t < w.t1 && ok; ++t, ++tile) {
                const int st = tile % stages, b = tile & 1, sb = tile % kScores;
                // (the loaders' own barrier too, for their scales and flags)
                ok = mbar_wait(smem_addr(&s.kv_full[st]), (tile / stages) & 1, status);
                const uint64_t missing = *reinterpret_cast<const volatile uint64_t *>(s.missing[st]);
                float2 rs[R / 8];
                auto read_scales = [&] {
#pragma unroll
                    for (int g8 = 0; g8 < R / 8; ++g8) {
                        const volatile float *at = &s.scales[st][8 * g8 + cq];
                        rs[g8] = make_float2(at[0], at[1]);
                    }
                };
                if constexpr (ROWS == kBits8)
                    read_scales();
                ok = ok && mbar_wait(smem_addr(&s.s_full[sb]), (tile / kScores) & 1, status);
                ok = __all_sync(~0u, ok);
                if (!ok)
                    break;
                tc_fence_after();
                constexpr int N = R / 2;  // values a thread
                float x[N];
#pragma unroll
                for (int i = 0; i < R / 32; ++i)
                    tmem_ld_16x256(my_lanes + (16u << 16) + sb * 64 + 32 * i, x + 16 * i);
                if constexpr (R % 32 == 16)
                    tmem_ld_16x256_half(my_lanes + (16u << 16) + sb * 64 + R - 16, x + N - 8);
                tmem_wait_ld();
                auto times_scales = [&](float2 v, int i) { return ROWS == kBits8 ? mul2(v, rs[i / 2]) : v; };  // v: x[2 i], x[2 i + 1]
                const bool masked = !whole || (t + 1) * R > all_see || missing;
                uint64_t see0 = ~0ull, see1 = ~0ull, poison = 0;
                if (masked) {
                    if (ROWS == kTma && (t + 1) * R > end) {
                        // Whole groups were copied: rows that no query sees may hold anything, and a weight of zero
                        // does not clear an infinity or NaN of theirs.
                        for (int i = (end - t * R) * (NK * 8) + tid; i < R * (NK * 8); i += 32 * kSoftWarps) {
                            const int row = i / (NK * 8), unit16 = i % (NK * 8);
                            *reinterpret_cast<uint4 *>(kv_mem + st * kTileBytes + (row >> 3) * kGroupBytes + (unit16 >> 3) * kGroupChunk +
                                                       (row & 7) * 128 + (unit16 & 7) * 16) = zero4();
                        }
                    }
                    if (all_see < end && (t + 1) * R > all_see) {
                        // Rows that some queries see and some do not: a weight of zero times an infinity or NaN would
                        // reach the queries that do not, so such a row is cleared, and the queries that see it get NaN.
                        const int row = tid >> 1;
                        uint8_t *mem = kv_mem + st * kTileBytes + (row >> 3) * kGroupBytes + (row & 7) * 128 + (tid & 1) * 64;
                        bool bad = false;
                        if (row < R && t * R + row >= all_see && t * R + row < end)
                            for (int ch = 0; ch < NK; ++ch)
#pragma unroll
                                for (int u = 0; u < 4; ++u) {
                                    const uint4 v = *reinterpret_cast<const uint4 *>(mem + ch * kGroupChunk + u * 16);
                                    bad |= nonfinite_bf16(v.x) || nonfinite_bf16(v.y) || nonfinite_bf16(v.z) || nonfinite_bf16(v.w);
                                }
                        if (ROWS == kBits8 && row < R)
                            bad |= !isfinite(s.scales[st][row]);
                        const uint32_t lanes = __ballot_sync(~0u, bad);
                        if (lanes >> (lane & ~1) & 3u) {
                            for (int ch = 0; ch < NK; ++ch)
#pragma unroll
                                for (int u = 0; u < 4; ++u)
                                    *reinterpret_cast<uint4 *>(mem + ch * kGroupChunk + u * 16) = zero4();
                            if (ROWS == kBits8)
                                s.scales[st][row] = 0.0f;
                        }
                        uint32_t bits = 0;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            bits |= (lanes >> (2 * i) & 3u) ? 1u << i : 0u;
                        // (two sets: a warp writes one again only after every warp has read it)
                        if (lane == 0) {
                            s.poison[flagged & 1][warp] = (uint16_t)bits;
                            mbar_arrive(smem_addr(&s.flags));
                        }
                        ok = mbar_wait(smem_addr(&s.flags), flagged & 1, status);
                        ok = __all_sync(~0u, ok);
                        if (!ok)
                            break;
                        poison = *reinterpret_cast<const volatile uint64_t *>(s.poison[flagged & 1]) >> cq;
                        ++flagged;
                        if constexpr (ROWS == kBits8)
                            read_scales();
                    }
                    auto mask = [&](int seen) {
                        const int lim = seen - t * R;
                        return (~missing & (lim <= 0 ? 0ull : lim >= 64 ? ~0ull : (1ull << lim) - 1)) >> cq;
                    };
                    see0 = mask(seen0);
                    see1 = mask(seen1);
                }
#pragma unroll
                for (int i = 0; i < N / 2; ++i) {
                    const float2 v = times_scales(make_float2(x[2 * i], x[2 * i + 1]), i);
                    x[2 * i] = v.x;
                    x[2 * i + 1] = v.y;
                }
                if (masked)
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const int bit = 8 * (i / 4) + (i & 1);
                        if (poison >> bit & 1)
                            x[i] = __int_as_float(0x7fffffff);
                        if (!(((i & 2) ? see1 : see0) >> bit & 1))
                            x[i] = -INFINITY;
                    }
                float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
                for (int i = 0; i < N; i += 4) {
                    t0 = fmaxf(t0, fmaxf(x[i], x[i + 1]));
                    t1 = fmaxf(t1, fmaxf(x[i + 2], x[i + 3]));
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    t0 = fmaxf(t0, __shfl_xor_sync(~0u, t0, o));
                    t1 = fmaxf(t1, __shfl_xor_sync(~0u, t1, o));
                }
                t0 *= f;
                t1 *= f;
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
                const float2 ff = splat(f), ref0 = splat(m0 == -INFINITY ? 0.0f : -m0), ref1 = splat(m1 == -INFINITY ? 0.0f : -m1);
                uint32_t pk[N / 2];  // of x[2 i], x[2 i + 1]
                float2 sum0 = splat(0.0f), sum1 = splat(0.0f);
#pragma unroll
                for (int i = 0; i < N / 2; ++i) {
                    const float2 y = fma2(make_float2(x[2 * i], x[2 * i + 1]), ff, (i & 1) ? ref1 : ref0);
                    float2 e = make_float2(exp2_fast(y.x), exp2_fast(y.y));
                    if (i & 1)
                        sum1 = add2(sum1, e);
                    else
                        sum0 = add2(sum0, e);
                    // (the scale of a row that the query does not see is finite: its weight stays 0)
                    pk[i] = f2_to_bf16x2(times_scales(e, i));
                }
                l0 += sum0.x + sum0.y;
                l1 += sum1.x + sum1.y;
                if (tile >= plan.p_buffers) {
                    // the buffer's last reader
                    const int pt = tile - plan.p_buffers;
                    ok = mbar_wait(smem_addr(&s.kv_empty[pt % stages]), (pt / stages) & 1, status);
                    ok = __all_sync(~0u, ok);
                    if (!ok)
                        break;
                }
                uint8_t *p_at = p_mem + (plan.p_buffers == 2 ? b : 0) * kQueryChunk + r0 * 128 + 2 * cq;
#pragma unroll
                for (int g8 = 0; g8 < R / 8; ++g8) {
                    uint8_t *at = p_at + ((g8 ^ (r0 & 7)) << 4);
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
            const bool done = !SHARED && w.t0 == 0 && w.t1 == w.nt;
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
            const bool live0 = r0 < item_rows, live1 = r0 + 8 < item_rows;
            if (done) {
                // the factor that turns O into the result
                auto finish = [&](int row, bool live, float m, float l) {
                    const float sink = live && p.sink ? __ldg(p.sink + p.by_heads.remainder(w.item() * kTile + row)) * kLog2E : -INFINITY;
                    const float top = fmaxf(m, sink), ref = top == -INFINITY ? 0.0f : top;
                    const float down = exp2_fast(m - ref), tot = l * down + exp2_fast(sink - ref);
                    if (live && p.lse && (lane & 3) == 0)
                        p.lse[out_row + row] = tot == 0.0f ? -INFINITY : (ref + log2f(tot)) * kLn2;
                    return tot == 0.0f ? 0.0f : down / tot;
                };
                const float inv0 = finish(r0, live0, m0, l0), inv1 = finish(r0 + 8, live1, m1, l1);
                uint16_t *dst = static_cast<uint16_t *>(p.out) + (out_row + r0) * p.v_dim + cq;
                for (int n = 0; n < p.v_dim; n += 64) {
                    float o[32];
                    if (w.t1 > w.t0) {
                        tmem_ld_16x256(my_lanes + n, o);
                        tmem_ld_16x256(my_lanes + n + 32, o + 16);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = 0.0f;
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        if (live0)
                            *reinterpret_cast<uint32_t *>(dst + n + 2 * i) = f2_to_bf16x2(make_float2(o[i] * inv0, o[i + 1] * inv0));
                        if (live1)
                            *reinterpret_cast<uint32_t *>(dst + 8 * p.v_dim + n + 2 * i) =
                                f2_to_bf16x2(make_float2(o[i + 2] * inv1, o[i + 3] * inv1));
                    }
                }
            } else {
                // (SHARED: of the pairs (item, block) in the order of the units, each has at least one number of the two one higher)
                const int64_t slot = SHARED ? (int64_t)w.index + c : 2 * (int64_t)c + (w.t0 == 0 ? 1 : 0);
                if constexpr (SHARED) {
                    if (w.index >= prefix.max_own)  // (there is room for every item of tokens that are each one request's)
                        continue;
                    if (tid == 0 && w.t0 == 0) {
                        const int2 own = own_of(prefix, w.r);
                        const int parts = w.nt == 0 ? 0 : holder(unit - 1 + (w.nt - w.t1), total, g) - c + 1;
                        prefix.items[w.index] = OwnItem{(int)out_row, item_rows, own.x > 0 ? own.y : -1, parts, (int)slot};
                    }
                    if (w.t1 == w.t0)
                        continue;
                }
                if ((lane & 3) == 0) {
                    plan.part_ml[slot * kTile + r0] = make_float2(m0, l0);
                    plan.part_ml[slot * kTile + r0 + 8] = make_float2(m1, l1);
                }
                if constexpr (SHARED)
                    for (int n = 0; n < p.v_dim; n += 64) {
                        float o[32];
                        tmem_ld_16x256(my_lanes + n, o);
                        tmem_ld_16x256(my_lanes + n + 32, o + 16);
                        tmem_wait_ld();
                        float *dst = plan.part_o + (slot * kTile + r0) * p.v_dim + n;
                        store_rows_16x256(dst, 8 * p.v_dim, o, live0, live1);
                        store_rows_16x256(dst + 32, 8 * p.v_dim, o + 16, live0, live1);
                    }
                float *dst = plan.part_o + (slot * kTile + r0) * p.v_dim + cq;
                for (int n = 0; !SHARED && n < p.v_dim; n += 64) {
                    float o[32];
                    tmem_ld_16x256(my_lanes + n, o);
                    tmem_ld_16x256(my_lanes + n + 32, o + 16);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        if (live0)
                            *reinterpret_cast<float2 *>(dst + n + 2 * i) = make_float2(o[i], o[i + 1]);
                        if (live1)
                            *reinterpret_cast<float2 *>(dst + 8 * p.v_dim + n + 2 * i) = make_float2(o[i + 2], o[i + 3]);
                    }
                }
                if (!SHARED && tid == 0 && (w.t0 == 0 || plan.helpers)) {
                    // the blocks of the item's first and last tile: its units around the segment's last one
                    const int first = w.t0 == 0 ? c : holder(unit - w.t1, total, g);
                    plan.joins[slot] = make_int4((int)out_row, item_rows, first, holder(unit - 1 + (w.nt - w.t1), total, g));
                }
            }
            tc_fence_before();
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------ matrix products
        // The warp stays together and one thread of it issues: the operands of tcgen05.mma are warp-uniform registers,
        // and a single thread running the loop alone would have each of them moved there, at some 100 cycles an MMA.
        const uint32_t tm = __shfl_sync(~0u, tmem, 0);
        const int stages_u = __shfl_sync(~0u, stages, 0);
        const uint64_t q_desc = mma_operand(smem_addr(q_mem), 16, 1024), p_desc = mma_operand(smem_addr(p_mem), 16, 1024);
        const uint64_t k_desc = mma_operand(smem_addr(kv_mem), 16, kGroupBytes);
        const uint64_t v_desc = mma_operand(smem_addr(kv_mem), kGroupChunk, kGroupBytes);
        constexpr uint32_t kTileStep = kTileBytes >> 4, kQueryStep = kQueryChunk >> 4, kChunkStep = kGroupChunk >> 4;
        constexpr uint32_t kSixteen = 2 * kGroupBytes >> 4;  // (of a descriptor's address) sixteen rows on
        constexpr uint32_t shape_s = mma_shape(kTile, R, false);
        auto scores = [&](int tile, int st, bool last) {  // S = Q K^T
            tc_fence_after();
            if (elect_one()) {
                const uint64_t k = k_desc + (uint32_t)st * kTileStep;
                const uint32_t d = tm + (16u << 16) + (tile % kScores) * 64;
#pragma unroll
                for (int ch = 0; ch < NK; ++ch)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma_bf16(d, q_desc + ch * kQueryStep + i * 2, k + ch * kChunkStep + i * 2, shape_s, ch > 0 || i > 0);
                mma_commit(smem_addr(&s.s_full[tile % kScores]));
                if (last)
                    mma_commit(smem_addr(&s.q_empty));
            }
            __syncwarp();
        };
        auto product = [&](int tile, int st, bool first) {  // O (+)= P V
            tc_fence_after();
            if (elect_one()) {
                const uint64_t v = v_desc + (uint32_t)st * kTileStep;
                const uint64_t pa = p_desc + (plan.p_buffers == 2 ? (tile & 1) * kQueryStep : 0);
                for (int n = 0; n < p.v_dim; n += 256) {
                    const uint32_t shape = mma_shape(kTile, min(256, p.v_dim - n), true);
#pragma unroll
                    for (int k = 0; k < R / 16; ++k)
                        mma_bf16(tm + n, pa + k * 2, v + (n / 64) * kChunkStep + k * kSixteen, shape, !first || k > 0);
                }
                mma_commit(smem_addr(&s.kv_empty[st]));
            }
            __syncwarp();
        };
        // i: the next tile to score, j <= i the next to multiply, at most kScores behind.  Whichever is ready goes first (a
        // tile's rows may wait for the product that frees their space), the product of the two: 250 against 248 us for
        // 608 tokens over 2048 rows of 512 columns, 335 against 305 us for rows of 576.
        int segment = 0, i = 0, i_st = 0, i_ph = 0, j = 0, j_st = 0;
        Walk<SHARED, R> w(p, prefix, s, units);
        while (ok && __shfl_sync(~0u, (int)w.next(), 0)) {
            const int n = __shfl_sync(~0u, w.t1 - w.t0, 0);
            if (n <= 0)
                continue;
            ok = mbar_wait(smem_addr(&s.q_full), segment++ & 1, status);
            ok = __all_sync(~0u, ok);
            const int first = j, end = j + n;
            while (ok && j < end) {
                const uint32_t kv_bar = smem_addr(&s.kv_full[i_st]), p_bar = smem_addr(&s.p_full[j & 1]);
                const uint32_t p_ph = (j >> 1) & 1;
                const bool may_score = i < end && i - j < kScores, may_multiply = j < i;
                bool score = false;
                uint64_t since = 0;
                for (uint32_t spins = 1;; ++spins) {
                    if (may_multiply && __all_sync(~0u, mbar_test(p_bar, p_ph)))
                        break;
                    score = may_score && __all_sync(~0u, mbar_test(kv_bar, i_ph));
                    if (score)
                        break;
                    if ((spins & 255u) == 0) {
                        const uint64_t now = __shfl_sync(~0u, global_ns(), 0);
                        since = since ? since : now;
                        if (now - since > kWaitLimitNs) {
                            if (lane == 0)
                                atomicCAS(status, 0u, kStatusTimeout);
                            ok = false;
                            break;
                        }
                    }
                }
                if (!ok)
                    break;
                if (score) {
                    scores(i, i_st, i + 1 == end);
                    ++i;
                    if (++i_st == stages_u) {
                        i_st = 0;
                        i_ph ^= 1;
                    }
                } else {
                    product(j, j_st, j == first);
                    ++j;
                    j_st = j_st + 1 == stages_u ? 0 : j_st + 1;
                }
            }
        }
        // nothing may be in flight when the block frees its memory, a wait that gave up included
        if (elect_one())
            mma_commit(smem_addr(&s.drained));
        __syncwarp();
        mbar_wait(smem_addr(&s.drained), 0, status);
        __syncwarp();
    } else if (ROWS != kTma || warp != kTmaWarp) {
        // ------------------------------------------------ queries, and rows, through registers
        const int lw = warp - (ROWS == kTma ? kTmaWarp : kMmaWarp) - 1;
        const uint8_t *cache = static_cast<const uint8_t *>(p.cache);
        int tile = 0, segment = 0;
        Walk<SHARED, R> w(p, prefix, s, units);
        while (ok && w.next()) {
            if (w.t1 <= w.t0)
                continue;
            const int item_rows = min(kTile, w.q.nq * p.n_heads - w.item() * kTile);
            {
                // 64 rows, four a warp at a time; the products S of the segment before have to be done
                constexpr int kTurns = kTile / (4 * kQueryArrivals);
                uint4 v[kTurns][NK];
#pragma unroll
                for (int i = 0; i < kTurns; ++i) {
                    const int row = (i * kQueryArrivals + lw) * 4 + (lane >> 3), flat = w.item() * kTile + row;
                    const uint8_t *src = static_cast<const uint8_t *>(p.q) + (lane & 7) * 16;
                    if (row < item_rows)
                        src += ((int64_t)(w.q.first + p.by_heads.quotient(flat)) * p.q_token_stride +
                                (int64_t)p.by_heads.remainder(flat) * p.q_head_stride) * 2;
#pragma unroll
                    for (int ch = 0; ch < NK; ++ch)
                        v[i][ch] = row < item_rows ? load_now(src + ch * 128) : zero4();
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
                    for (int ch = 0; ch < NK; ++ch)
                        *reinterpret_cast<uint4 *>(dst + ch * kQueryChunk) = v[i][ch];
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&s.q_full));
            }
            if constexpr (ROWS != kTma) {
                // Groups of eight rows, counted through the block's tiles; the warp takes every eighth.  A lane finds the
                // page of one row (lane % 8) a turn ahead; 8-bit rows are fetched a turn ahead too (twice the registers
                // would not do for bf16 rows).
                const int end = visible(p, w.q, last_token(p, w.q, w.item()));
                const int32_t *table = w.table();
                const int n_groups = (w.t1 - w.t0) * kGroups;
                constexpr bool kAhead = ROWS == kBits8;
                constexpr int kParts = ROWS == kBits8 ? 1 : 2;  // 8-bit: lane / 4 is the row, else lane / 8 and + 4
                auto row_of = [&](int i) { return w.t0 * R + i * 8 + (lane & 7); };
                auto look_up = [&](int i) { return i < n_groups && row_of(i) < end ? load_now(table + p.by_page.quotient(row_of(i))) : 0; };
                struct Fetched {
                    uint4 v[kParts][NK];
                    float scale;
                    uint32_t missing;
                };
                auto fetch = [&](int i, int page, Fetched &f8) {
                    const bool need = i < n_groups && row_of(i) < end, found = page >= 0 && page < p.n_pages;
                    const int64_t slot = need && found ? (int64_t)page * p.page_size + p.by_page.remainder(row_of(i)) : -1;
                    f8.missing = __ballot_sync(~0u, need && !found) & 0xffu;
#pragma unroll
                    for (int h = 0; h < kParts; ++h) {
                        const int64_t at = __shfl_sync(~0u, slot, ROWS == kBits8 ? lane >> 2 : (lane >> 3) + 4 * h);
                        const uint8_t *src = ROWS == kBits8 ? cache + at * p.cache_stride + (lane & 3) * 16
                                                            : cache + at * p.cache_stride * 2 + (lane & 7) * 16;
#pragma unroll
                        for (int ch = 0; ch < NK; ++ch)
                            f8.v[h][ch] = at >= 0 ? load_now(src + ch * (ROWS == kBits8 ? 64 : 128)) : zero4();
                    }
                    f8.scale = ROWS == kBits8 && slot >= 0 ? __ldg(p.row_scales + slot) : 0.0f;
                };
                auto put = [&](int i, const Fetched &f8) {
                    const int mine = tile + i / kGroups, gr = i % kGroups, st = mine % stages;
                    if (mine >= stages) {
                        ok = mbar_wait(smem_addr(&s.kv_empty[st]), (mine / stages - 1) & 1, status);
                        ok = __all_sync(~0u, ok);
                        if (!ok)
                            return;
                    }
                    uint8_t *dst = kv_mem + st * kTileBytes + gr * kGroupBytes;
                    if constexpr (ROWS == kBits8) {
                        if (lane < 8)
                            s.scales[st][gr * 8 + lane] = f8.scale;
                        const int r = lane >> 2, quarter = lane & 3;  // 16 of a chunk's 64 columns
#pragma unroll
                        for (int ch = 0; ch < NK; ++ch)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const uint32_t a = u ? f8.v[0][ch].z : f8.v[0][ch].x, e = u ? f8.v[0][ch].w : f8.v[0][ch].y;
                                *reinterpret_cast<uint4 *>(dst + ch * kGroupChunk + r * 128 + (((2 * quarter + u) ^ r) << 4)) =
                                    make_uint4(bf16x2_of_e4m3x2(a & 0xffffu), bf16x2_of_e4m3x2(a >> 16),
                                               bf16x2_of_e4m3x2(e & 0xffffu), bf16x2_of_e4m3x2(e >> 16));
                            }
                    } else {
#pragma unroll
                        for (int h = 0; h < kParts; ++h) {
                            const int r = (lane >> 3) + 4 * h;
#pragma unroll
                            for (int ch = 0; ch < NK; ++ch)
                                *reinterpret_cast<uint4 *>(dst + ch * kGroupChunk + r * 128 + (((lane & 7) ^ r) << 4)) = f8.v[h][ch];
                        }
                    }
                    if (lane == 0)
                        s.missing[st][gr] = (uint8_t)f8.missing;
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_addr(&s.kv_full[st]));
                };
                int i = (lw - tile * kGroups) & (kLoadWarps - 1);
                int page = look_up(i);
                Fetched a, e;
                if constexpr (kAhead) {
                    fetch(i, page, a);
                    page = look_up(i + kLoadWarps);
                    for (; ok && i < n_groups; i += 2 * kLoadWarps) {
                        fetch(i + kLoadWarps, page, e);
                        page = look_up(i + 2 * kLoadWarps);
                        put(i, a);
                        if (!ok || i + kLoadWarps >= n_groups)
                            break;
                        fetch(i + 2 * kLoadWarps, page, a);
                        page = look_up(i + 3 * kLoadWarps);
                        put(i + kLoadWarps, e);
                    }
                } else {
                    for (; ok && i < n_groups; i += kLoadWarps) {
                        fetch(i, page, a);
                        page = look_up(i + kLoadWarps);
                        put(i, a);
                    }
                }
                tile += w.t1 - w.t0;
            }
        }
    } else if constexpr (ROWS == kTma) {
        // ------------------------------------------------ rows by TMA, in groups of eight
        const uint32_t kv_smem = smem_addr(kv_mem);
        const int none = (int)(p.n_pages * p.page_size / 8);  // a group past the end reads as zeros
        const int copies = kGroups / plan.box_groups;
        uint32_t dirty = 0;  // stages whose flags are not all clear
        int tile = 0;
        Walk<SHARED, R> w(p, prefix, s, units);
        while (ok && w.next()) {
            const int end = visible(p, w.q, last_token(p, w.q, w.item()));
            const int32_t *table = w.table();
            // lane % 8 finds the page of one of a tile's groups, a tile ahead
            auto needed = [&](int t) { return t < w.t1 && (lane & 7) < kGroups && t * R + (lane & 7) * 8 < end; };
            auto look_up = [&](int t) { return needed(t) ? load_now(table + p.by_page.quotient(t * R + (lane & 7) * 8)) : 0; };
            int next = look_up(w.t0);
            for (int t = w.t0; t < w.t1; ++t, ++tile) {
                const int st = tile % stages;
                const bool need = needed(t), found = next >= 0 && next < p.n_pages;
                const uint32_t missing = __ballot_sync(~0u, need && !found) & 0xffu;
                const int at = need && found ? (next * p.page_size + (int)p.by_page.remainder(t * R + (lane & 7) * 8)) >> 3 : none;
                next = look_up(t + 1);
                // all that can be is found before the wait
                const uint32_t bar = smem_addr(&s.kv_full[st]), dst = kv_smem + st * kTileBytes;
                const bool plain = !missing && (t + 1) * R <= end;  // runs of groups that lie together
                const int first = __shfl_sync(~0u, at, plain ? (lane & 7) * plan.box_groups & 7 : lane & 7);
                if (tile >= stages) {
                    ok = mbar_wait(smem_addr(&s.kv_empty[st]), (tile / stages - 1) & 1, status);
                    ok = __all_sync(~0u, ok);
                    if (!ok)
                        break;
                }
                if (missing || dirty >> st & 1) {
                    if (lane < 8)
                        s.missing[st][lane] = missing >> lane & 1 ? 0xff : 0;
                    dirty = missing ? dirty | 1u << st : dirty & ~(1u << st);
                    __syncwarp();
                }
                if (lane == 0)
                    mbar_arrive_expect_tx(bar, kTileBytes);
                __syncwarp();
                if (plain ? lane < copies : lane < kGroups)
                    tma_load_4d(dst + lane * (plain ? plan.box_groups : 1) * kGroupBytes, plain ? &boxes : &groups, 0, 0, 0, first, bar);
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
    if constexpr (SHARED)
        pdl_wait();
}

// Joins the parts of the items that cross block boundaries, a warp a row.  Part k of n is slot 1 of the item's first block
// (k = 0) or slot 0 of the block k further on.  The blocks of part 0 join them, four loads a lane under way.  Where there
// are few items (plan.helpers) the blocks of all parts join those of more than four: part i takes the row's columns, in
// units of 32, from unit i on in steps of n, and reads four parts of a unit at once, eight lanes each (one request of
// 16384 rows, 85 parts: 41.8 us with part 0 alone, 27.4 so; 16 items of ten parts: 42.0 and 48.3).  Sums run over the
// parts in a fixed order.  Bound by the latency of three dependent reads and by the launches of blocks that find no part.
template <bool HELPERS> __global__ void __launch_bounds__(128) latent_join_kernel(const AttnParams p, const MmaPlan plan)
{
    pdl_wait();
    pdl_trigger();
    // the parts 0 first: theirs are the longest blocks
    const int blocks = plan.blocks, slot = blockIdx.x < blocks ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x - blocks);
    const int lane = threadIdx.x & 31, row = blockIdx.y * 4 + (threadIdx.x >> 5);
    const int4 j = plan.joins[slot];
    const int c = j.z, n = j.w - c + 1, mine = slot / 2 - c, units = p.v_dim / 32;
    const bool shared = HELPERS && n > 4;
    if (row >= j.y || mine >= (shared ? units : 1))
        return;
    const int64_t out_row = (int64_t)j.x + row;
    const float sink = p.sink ? __ldg(p.sink + p.by_heads.remainder((uint32_t)out_row)) * kLog2E : -INFINITY;
    auto part = [&](int k) { return (2 * (int64_t)(c + k) + (k == 0 ? 1 : 0)) * kTile + row; };
    float top = sink;
    for (int k = lane; k < n; k += 32)
        top = fmaxf(top, plan.part_ml[part(k)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    const float ref = top == -INFINITY ? 0.0f : top;
    float tot = lane == 0 ? exp2_fast(sink - ref) : 0.0f, weight = 0.0f;
    for (int k = lane; k < n; k += 32) {
        const float2 ml = plan.part_ml[part(k)];
        weight = exp2_fast(ml.x - ref);
        tot = fmaf(weight, ml.y, tot);
    }
#pragma unroll
    for (int i = 16; i; i >>= 1)
        tot += __shfl_xor_sync(~0u, tot, i);
    const float inv = tot == 0.0f ? 0.0f : 1.0f / tot;
    auto add = [](float4 &o, float w, const float *src) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(src));
        o.x = fmaf(w, v.x, o.x);
        o.y = fmaf(w, v.y, o.y);
        o.z = fmaf(w, v.z, o.z);
        o.w = fmaf(w, v.w, o.w);
    };
    auto write = [&](int col, const float4 &o) {
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + out_row * p.v_dim + col) =
            make_uint2(f2_to_bf16x2(make_float2(o.x * inv, o.y * inv)), f2_to_bf16x2(make_float2(o.z * inv, o.w * inv)));
    };
    if (!HELPERS || !shared) {
        float4 o[4] = {};
#pragma unroll 2
        for (int k = 0; k < n; ++k) {
            const float w = n <= 32 ? __shfl_sync(~0u, weight, k & 31) : exp2_fast(plan.part_ml[part(k)].x - ref);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (lane * 4 + 128 * i < p.v_dim)
                    add(o[i], w, plan.part_o + part(k) * p.v_dim + lane * 4 + 128 * i);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane * 4 + 128 * i < p.v_dim)
                write(lane * 4 + 128 * i, o[i]);
    } else {
        const int group = lane >> 3;
        for (int u = mine; u < units; u += n) {
            const int col = u * 32 + (lane & 7) * 4;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int k = group; k < n; k += 4)
                add(o, exp2_fast(plan.part_ml[part(k)].x - ref), plan.part_o + part(k) * p.v_dim + col);
#pragma unroll
            for (int x = 8; x < 32; x <<= 1) {
                o.x += __shfl_xor_sync(~0u, o.x, x);
                o.y += __shfl_xor_sync(~0u, o.y, x);
                o.z += __shfl_xor_sync(~0u, o.z, x);
                o.w += __shfl_xor_sync(~0u, o.w, x);
            }
            if (group == 0)
                write(col, o);
        }
    }
    if (p.lse && lane == 0 && mine == 0)
        p.lse[out_row] = tot == 0.0f ? -INFINITY : (ref + log2f(tot)) * kLn2;
}

template <bool SHARED, Rows ROWS, int NK, int R>
cudaError_t go(const AttnParams &p, const MmaPlan &plan, const Prefix<SHARED> &prefix, unsigned *status, cudaStream_t st)
{
    auto kern = latent_mma_kernel<SHARED, ROWS, NK, R>;
    cudaError_t e = allow_max_smem(reinterpret_cast<const void *>(kern));
    CUtensorMap boxes = {}, groups = {};
    if (ROWS == kTma && e == cudaSuccess && p.width > 0) {
        const int64_t rows = p.n_pages * p.page_size;
        e = make_tensor_map_groups(&groups, p.cache, rows, NK, p.cache_stride, 1);
        if (e == cudaSuccess)
            e = make_tensor_map_groups(&boxes, p.cache, rows, NK, p.cache_stride, plan.box_groups);
    }
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = st;
    cfg.gridDim = dim3(plan.blocks);
    cfg.blockDim = dim3(kThreadsOf<ROWS, NK>);
    cfg.dynamicSmemBytes = plan.smem;
    e = cudaLaunchKernelEx(&cfg, kern, p, plan, prefix, boxes, groups, status);
    if (e != cudaSuccess || SHARED)
        return e;
    cfg.gridDim = dim3((plan.helpers ? 2 : 1) * plan.blocks, kTile / 4);
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    return plan.helpers ? cudaLaunchKernelEx(&cfg, latent_join_kernel<true>, p, plan)
                        : cudaLaunchKernelEx(&cfg, latent_join_kernel<false>, p, plan);
}

// Dynamic shared memory of a block: what an SM has for one, or half of it, less the block's own.
constexpr size_t smem_limit(Rows how, int nk) { return (per_sm(how, nk) == 2 ? 113 : 227) * 1024 - sizeof(Shared); }

constexpr size_t fixed_of(int nk) { return (size_t)(nk + 1) * kQueryChunk + 1024; }  // queries, P, alignment

constexpr int stages_of(Rows how, int nk, int rows)
{
    return (int)((smem_limit(how, nk) - fixed_of(nk)) / ((size_t)nk * rows * 128));
}

// Rows of a tile: the tensor core wants wide tiles, the loads want three tiles in flight; so 64 where three fit beside
// the queries, else 48 (512 columns: a decode step of 64 requests 94.6 us against 97.5 with two tiles of 64 rows), else
// (576 columns) two of 64 (608 tokens over 2048 rows 260 us against 305 with four of 32, which cost the tensor core as
// much as 40 would).
constexpr int rows_of(Rows how, int nk) { return stages_of(how, nk, 64) < 3 && stages_of(how, nk, 48) >= 3 ? 48 : 64; }

Rows rows_how(const AttnParams &p)
{
    return p.cache_dtype == CSA_DTYPE_E4M3 ? kBits8 : p.page_size % 8 == 0 ? kTma : kRegisters;
}

MmaPlan make_plan(const AttnParams &p, int num_sms)
{
    MmaPlan m{};
    const Rows how = rows_how(p);
    const int nk = p.head_dim / 64, rows = rows_of(how, nk), fit = stages_of(how, nk, rows);
    m.stages = fit > kMaxStages ? kMaxStages : fit;
    m.smem = fixed_of(nk) + (size_t)m.stages * nk * rows * 128;
    m.p_buffers = m.smem + kQueryChunk <= smem_limit(how, nk) ? 2 : 1;
    m.smem += (m.p_buffers - 1) * kQueryChunk;
    // the larger copy: the most groups that divide both the tile and the page
    for (m.box_groups = rows / 8; m.box_groups > 1 && (p.page_size % (8 * m.box_groups) || (rows / 8) % m.box_groups); --m.box_groups) {}
    // room for what cuts the work; one block an SM (it owns the tensor memory): more than half of the shared memory
    constexpr size_t least = 1024 + (kMaxRequests + 4) * sizeof(int) + kKept * sizeof(Request);
    static_assert(least < smem_limit(kTma, 1), "");
    const size_t floor_bytes = per_sm(how, nk) == 2 ? least : 116 * 1024;
    m.smem = m.smem < floor_bytes ? floor_bytes : m.smem;
    m.tmem_columns = p.v_dim > 256 ? 512 : 256;  // O below, the S tiles above
    m.blocks = num_sms * per_sm(how, nk);
    m.helpers = 16 * ((p.n_tokens * p.n_heads) / kTile + p.n_req) < m.blocks;  // (at least a bound of the items)
    return m;
}

template <bool SHARED, int NK>
cudaError_t go_rows(const AttnParams &p, const MmaPlan &m, const Prefix<SHARED> &prefix, unsigned *status, cudaStream_t st)
{
    switch (rows_how(p)) {
    case kTma: return go<SHARED, kTma, NK, rows_of(kTma, NK)>(p, m, prefix, status, st);
    case kRegisters: return go<SHARED, kRegisters, NK, rows_of(kRegisters, NK)>(p, m, prefix, status, st);
    default: return go<SHARED, kBits8, NK, rows_of(kBits8, NK)>(p, m, prefix, status, st);
    }
}

// LEAST: the narrowest rows that there are kernels for, in units of 64 columns.
template <bool SHARED, int LEAST>
cudaError_t launch_mma(const AttnParams &p, const Prefix<SHARED> &prefix, void *workspace, int num_sms, unsigned *status, cudaStream_t st)
{
    MmaPlan m = make_plan(p, num_sms);
    if constexpr (SHARED) {
        m.part_o = prefix.own_o;
        m.part_ml = prefix.own_ml;
    } else {
        m.part_o = static_cast<float *>(workspace);
        m.part_ml = reinterpret_cast<float2 *>(m.part_o + (size_t)m.blocks * 2 * kTile * p.v_dim);
        m.joins = reinterpret_cast<int4 *>(m.part_ml + (size_t)m.blocks * 2 * kTile);
    }
    switch (p.head_dim / 64) {
    case 1:
        if constexpr (LEAST <= 1)
            return go_rows<SHARED, 1>(p, m, prefix, status, st);
        return cudaErrorInvalidValue;
    case 2: return go_rows<SHARED, 2>(p, m, prefix, status, st);
    case 3: return go_rows<SHARED, 3>(p, m, prefix, status, st);
    case 4: return go_rows<SHARED, 4>(p, m, prefix, status, st);
    case 5: return go_rows<SHARED, 5>(p, m, prefix, status, st);
    case 6: return go_rows<SHARED, 6>(p, m, prefix, status, st);
    case 7: return go_rows<SHARED, 7>(p, m, prefix, status, st);
    case 8: return go_rows<SHARED, 8>(p, m, prefix, status, st);
    case 9: return go_rows<SHARED, 9>(p, m, prefix, status, st);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

// csa_latent_behind.cu compiles this file again for requests behind a prefix.
#ifndef CSA_BEHIND_PREFIX
bool latent_mma_supported(const AttnParams &p)
{
    return on_tensor_cores(p.head_dim, p.v_dim);
}

size_t latent_mma_workspace(const AttnParams &p, int num_sms)
{
    const MmaPlan m = make_plan(p, num_sms);
    return (size_t)m.blocks * 2 * (kTile * ((size_t)p.v_dim * sizeof(float) + sizeof(float2)) + sizeof(int4));
}

cudaError_t launch_latent_mma(const AttnParams &p, void *workspace, int num_sms, unsigned *status, cudaStream_t st)
{
    return launch_mma<false, 1>(p, NoPrefix{}, workspace, num_sms, status, st);
}
#endif

}  // namespace csa
