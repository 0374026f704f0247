// Attention for a batch whose requests share prefixes, in two parts that are joined by their sums:
//
//   s_j = scale q.k_j;   over any set A of rows:  m_A >= max s_j - 8 log 2,  l_A = sum e^(s_j - m_A),  O_A = sum e^(s_j - m_A) v_j
//   out = sum_A e^(m_A - m) O_A / (sum_A e^(m_A - m) l_A + e^(sink - m))
//
// The prefix's rows are read once for all (token, head) pairs of the group, as one matrix product after another with the group's
// queries as rows (latent_pair_kernel here); the requests' own rows by the kernel that attends request by request
// (csa_latent_mma.cu, compiled for them in csa_latent_behind.cu).  Both leave parts (O, m, l), which shared_join_kernel joins in a
// fixed order.  Rows that some token of the group does not see, or that do not fill a page, count as own rows, so the prefix part
// has no mask but its last tile's end.
//
// A prefix part is bound by the tensor cores: with 64 query rows a block, as the attention by requests has them, an MMA runs at half
// the rate (O of 128 rows x 512 columns in fp32 would fill tensor memory).  So two blocks work as a pair (cta_group::2): an
// item is 128 query rows, 64 a block, in all 128 lanes of each block's tensor memory.  For each tile of 128 cache rows:
//
//   S = Q K^T          128 x 128: each block holds 64 query rows and loads 64 of the tile's rows
//   P = exp2(S f - m)  a thread has one query row and a quarter of the tile's columns
//   O += P V           128 x v_dim: each block loads half of the value columns of all 128 rows
//
// so a block loads 128 KB for the 33.6 MFLOP of the two at 512 columns, in units of 64 rows x up to two chunks of 64 columns (16
// KB), through a ring for K and one for V (four units each there; seven in all for rows of 576).  S, P and O of neighbouring tiles overlap: S runs up to two tiles ahead, P has two buffers.  The running
// reference m is raised only when a logit exceeds it by 2^8, so O is rarely touched outside the tensor core, and P stays below 2^8.
//
// 32768 query rows over 8192 rows of 512 columns (512 requests of 64 heads): some 300 us of the call's 411, 1.8 PFLOP/s, 2500 cycles a tile of which the
// tensor core needs 2048 (482 us with one warp that issued MMAs and waited for every unit, four of
// exponentials, one that copied, and arrivals that ordered global memory too).
//
// Work is cut evenly over the pairs as in csa_latent_cuts.h.  Rows that are not bf16 in pages of whole groups of eight are first
// widened to bf16 (8-bit values exactly; their scales stay apart) into an image of the prefix.
#include <cuda.h>
#include <cuda_fp8.h>

#include "csa_launch.h"
#include "csa_serving_launch.h"
#include "csa_shared.cuh"
#include "csa_tcgen05.cuh"

namespace csa {
namespace {

constexpr int kHalf = 64;                 // query rows of a block
constexpr int kQueryChunk = kHalf * 128;  // bytes of 64 columns of a block's queries
constexpr int kSoftWarps = 8, kScoreWarp = 8, kValueWarp = 9, kCopyWarp = 10, kCopyWarps = 4, kQueryWarp = 14, kQueryWarps = 2;
constexpr int kThreads = 32 * (kQueryWarp + kQueryWarps);
constexpr int kMaxSlots = 16;
constexpr int kBatch = 2;  // units that an MMA warp waits for at once
constexpr float kLog2E = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kRaise = 8.0f;  // log2 of how far a logit may exceed the reference

struct PairPlan {
    int nk;           // chunks of 64 columns of a row
    int vch;          // chunks of a block's half of the value columns
    int cw;           // chunks of a unit
    int k_slots, v_slots;  // units in the rings of K and V
    int box_groups;   // groups of eight rows of the larger copy
    size_t smem;
};

struct PairShared {
    uint64_t kv_full[kMaxSlots], kv_empty[kMaxSlots], s_full[2], p_full[2], pv_done[2], q_full, q_empty, drained;
    uint32_t tmem;
    int g, m, off, base;  // where the pair's units begin: group, item, unit of the item, items before the group
    long long total;
    float exchange[32 * kSoftWarps];
};

// A group's items, held to the parts that there is room for (only groups that overlap have more).
__device__ __forceinline__ int items_of(const SharedPlan &s, const GroupInfo &q, int base) { return min(q.items, max(s.max_items - base, 0)); }

// The pair's segments, walked alike by every role of both blocks.
struct PairWalk {
    const SharedPlan &s;
    GroupInfo q;
    int g, m, off, base, items;
    long long left;
    int t0, t1;
    __device__ PairWalk(const SharedPlan &s_, const PairShared &at, long long units) : s(s_), g(at.g), m(at.m), off(at.off), base(at.base), left(units)
    {
        if (left > 0) {
            q = s.groups[g];
            items = items_of(s, q, base);
        }
    }
    // the next segment: tiles [t0, t1) of item m - 1 of group g
    __device__ bool next()
    {
        while (left > 0) {
            while (m >= items) {
                base += items;
                if (++g >= s.n_groups)
                    return false;
                m = 0;
                q = s.groups[g];
                items = items_of(s, q, base);
            }
            const Segment x = segment_of(q.tiles, off, left, kPairHead);
            t0 = x.t0;
            t1 = x.t1;
            left -= x.take;
            off = 0;
            ++m;
            if (t1 > t0)
                return true;
        }
        return false;
    }
    __device__ int item() const { return m - 1; }
};

// CW: chunks of a unit, a constant so that an MMA's operands are a base and constants
template <bool BITS8, int CW>
__global__ void __launch_bounds__(kThreads, 1)
latent_pair_kernel(const AttnParams p, const SharedPlan s, const PairPlan plan, const __grid_constant__ CUtensorMap boxes,
                   const __grid_constant__ CUtensorMap groups, unsigned *status)
{
    extern __shared__ uint8_t raw[];
    __shared__ PairShared sh;
    uint8_t *mem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    constexpr int cw = CW, group_bytes = cw * 1024, unit_bytes = 8 * group_bytes;
    const int nk = plan.nk;
    uint8_t *q_mem = mem, *p_mem = q_mem + nk * kQueryChunk, *kv_mem = p_mem + 4 * kQueryChunk;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const int c = blockIdx.x / 2;

    if (tid == 0) {
        for (int i = 0; i < plan.k_slots + plan.v_slots; ++i) {
            mbar_init(smem_addr(&sh.kv_full[i]), 1);
            mbar_init(smem_addr(&sh.kv_empty[i]), 1);
        }
        // (two each, by the tile's parity: a block may be a tile ahead of the other)
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sh.s_full[i]), 1);
            mbar_init(smem_addr(&sh.p_full[i]), 2 * kSoftWarps);
            mbar_init(smem_addr(&sh.pv_done[i]), 1);
        }
        mbar_init(smem_addr(&sh.q_full), 2 * kQueryWarps);
        mbar_init(smem_addr(&sh.q_empty), 1);
        mbar_init(smem_addr(&sh.drained), 2);
        mbar_init_fence();
    }
    pdl_wait();
    pdl_trigger();
    if (warp == kScoreWarp)
        tmem_alloc_pair(smem_addr(&sh.tmem), 512);
    if (warp == 0) {
        // ---- where the pair's units begin: two passes over the groups, 32 at a time
        long long total = 0, from = 0;
        for (int pass = 0; pass < 2; ++pass) {
            int base = 0;
            long long units = 0;
            for (int at = 0; at < s.n_groups; at += 32) {
                const int g = at + lane;
                GroupInfo q{};
                if (g < s.n_groups)
                    q = s.groups[g];
                int a = q.items;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int u = __shfl_up_sync(~0u, a, o);
                    if (lane >= o)
                        a += u;
                }
                const int before = min(base + a - q.items, s.max_items), items = items_of(s, q, before);
                const long long mine = (long long)items * (q.tiles + kPairHead);
                long long b = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long u = __shfl_up_sync(~0u, b, o);
                    if (lane >= o)
                        b += u;
                }
                const long long first = units + b - mine;
                if (pass == 1) {
                    if (from >= first && from < first + mine) {
                        const int each = q.tiles + kPairHead;
                        sh.g = g;
                        sh.m = (int)((from - first) / each);
                        sh.off = (int)((from - first) % each);
                        sh.base = before;
                    }
                    if (blockIdx.x == 0 && g < s.n_groups)
                        s.sums[g] = GroupSums{first, before, items};
                }
                base = min(base + __shfl_sync(~0u, a, 31), s.max_items);
                units += __shfl_sync(~0u, b, 31);
            }
            if (pass == 0) {
                total = units;
                const int n = sharing(total, s.clusters);
                from = c < n ? cut(total, c, n) : total;
            }
        }
        if (lane == 0) {
            sh.total = total;
            if (blockIdx.x == 0)
                *s.total = total;
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_barrier();  // the other block's barriers are initialised too
    tc_fence_after();
    const long long total = sh.total;
    const int n_sharing = sharing(total, s.clusters);
    const long long units = c < n_sharing ? cut(total, c + 1, n_sharing) - cut(total, c, n_sharing) : 0;
    const uint32_t tmem = sh.tmem;
    const int v_half = plan.vch * 64;
    bool ok = true;

    if (warp < kSoftWarps) {
        // ------------------------------------------------ exponentials and output
        // this thread's query row, and a quarter of a tile's columns: 32 of the half that its lanes have
        const int row = tid & 63, half = tid >> 6 & 1, part = warp >> 2;
        const uint32_t my_lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16), p_full0 = at_rank(smem_addr(&sh.p_full[0]), 0);
        const float f = p.scale * kLog2E;
        int tile = 0;
        PairWalk w(s, sh, units);
        // (every thread comes to the block's barriers, after a wait that gave up too)
        auto wait = [&](uint64_t *bar, int phase) {
            ok = ok && mbar_wait(smem_addr(bar), phase & 1, status);
            ok = __all_sync(~0u, ok);
        };
        while (ok && w.next()) {
            const int rows = min(kPairRows, w.q.rows - w.item() * kPairRows);
            const float *scales = BITS8 ? s.image_scales + (int64_t)w.g * s.image_rows + half * 64 + part * 32 : nullptr;
            float m = -INFINITY, l = 0.0f;
            for (int t = w.t0; t < w.t1; ++t, ++tile) {
                wait(&sh.s_full[tile & 1], tile >> 1);
                tc_fence_after();
                float x[32];
                tmem_ld_32x32(my_lanes + 256 + (tile & 1) * 64 + part * 32, x);
                tmem_wait_ld();
                if constexpr (BITS8)
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 v = __ldg(reinterpret_cast<const float4 *>(scales + t * kPairRows + i));
                        x[i] *= v.x, x[i + 1] *= v.y, x[i + 2] *= v.z, x[i + 3] *= v.w;
                    }
                const int lim = w.q.shared - t * kPairRows - half * 64 - part * 32;
                if (lim < 32)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        x[i] = i < lim ? x[i] : -INFINITY;
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < 32; i += 2)
                    top = fmaxf(top, fmaxf(x[i], x[i + 1]));
                top *= f;
                if (!named_barrier_and(1, 32 * kSoftWarps, ok && !(top > m + kRaise))) {
                    sh.exchange[tid] = top;
                    if (!named_barrier_and(2, 32 * kSoftWarps, ok)) {
                        ok = false;
                        break;
                    }
                    top = fmaxf(fmaxf(sh.exchange[row], sh.exchange[row + 64]), fmaxf(sh.exchange[row + 128], sh.exchange[row + 192]));
                    const bool up = top > m + kRaise;  // (-inf > -inf is false)
                    const float down = up ? exp2_fast(m - top) : 1.0f;
                    m = up ? top : m;
                    l *= down;
                    if (t > w.t0) {
                        wait(&sh.pv_done[(tile - 1) & 1], (tile - 1) >> 1);
                        if (ok) {
                            tc_fence_after();
                            for (int n = part * 32; n < v_half; n += 64) {
                                float o[32];
                                tmem_ld_32x32(my_lanes + n, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    o[i] *= down;
                                tmem_st_32x32(my_lanes + n, o);
                            }
                            tmem_wait_st();
                        }
                    }
                }
                const float2 ff = splat(f), ref = splat(m == -INFINITY ? 0.0f : -m);
                uint32_t pk[16];
                float2 sum = splat(0.0f);
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    float4 v = make_float4(1.f, 1.f, 1.f, 1.f);
                    if constexpr (BITS8)
                        v = __ldg(reinterpret_cast<const float4 *>(scales + t * kPairRows + i));
#pragma unroll
                    for (int k = 0; k < 4; k += 2) {
                        const float2 y = fma2(make_float2(x[i + k], x[i + k + 1]), ff, ref);
                        float2 e = make_float2(exp2_fast(y.x), exp2_fast(y.y));
                        sum = add2(sum, e);
                        if constexpr (BITS8)
                            e = mul2(e, k ? make_float2(v.z, v.w) : make_float2(v.x, v.y));
                        pk[(i + k) / 2] = f2_to_bf16x2(e);
                    }
                }
                l += sum.x + sum.y;
                if (tile > 1)
                    wait(&sh.pv_done[tile & 1], (tile - 2) >> 1);  // the buffer's last reader
                uint8_t *dst = p_mem + ((tile & 1) * 2 + half) * kQueryChunk + row * 128;
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    *reinterpret_cast<uint4 *>(dst + (((part * 4 + u) ^ (row & 7)) << 4)) =
                        make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster(p_full0 + (tile & 1) * 8);
            }
            // ---- the part to the workspace
            if (ok)
                wait(&sh.pv_done[(tile - 1) & 1], (tile - 1) >> 1);
            sh.exchange[tid] = l;
            ok = named_barrier_and(3, 32 * kSoftWarps, ok);
            if (!ok)
                break;
            tc_fence_after();
            const int64_t slot = ((int64_t)w.base + w.item() + c) * kPairRows + rank * kHalf;
            if (tid < kHalf)
                s.part_ml[slot + row] =
                    make_float2(m, (sh.exchange[row] + sh.exchange[row + 64]) + (sh.exchange[row + 128] + sh.exchange[row + 192]));
            for (int sub = 0; sub < 2; ++sub) {
                const int r = (warp & 1) * 32 + sub * 16 + lane / 4, left = rows - (int)rank * kHalf;
                float *dst = s.part_o + (slot + r) * p.v_dim + half * v_half;
                for (int n = part * 32; n < v_half; n += 64) {
                    float o[16];
                    tmem_ld_16x256(my_lanes + ((uint32_t)(sub * 16) << 16) + n, o);
                    tmem_wait_ld();
                    store_rows_16x256(dst + n, 8 * p.v_dim, o, r < left, r + 8 < left);
                }
            }
            tc_fence_before();
        }
    } else if (warp <= kValueWarp) {
        // ------------------------------------------------ matrix products, issued by the even block
        // Two warps, one for S and one for O: between its products each spends as long again on waits and loops, while the other's
        // run (one warp for both: 3050 cycles a tile).  Units are taken kBatch at a time for the same reason.  Each has a ring of its
        // own: a barrier's parity says that a phase is over only to who knows that the one before is, as a ring's only reader does.
        if (rank == 0) {
            const uint32_t tm = __shfl_sync(~0u, tmem, 0);
            const uint64_t q_desc = mma_operand(smem_addr(q_mem), 16, 1024), p_desc = mma_operand(smem_addr(p_mem), 16, 1024);
            const uint64_t k_desc = mma_operand(smem_addr(kv_mem), 16, group_bytes), v_desc = mma_operand(smem_addr(kv_mem), 1024, group_bytes);
            constexpr uint32_t unit_step = unit_bytes >> 4, sixteen = 2 * group_bytes >> 4;
            constexpr uint32_t kQueryStep = kQueryChunk >> 4, kChunkStep = 1024 >> 4;
            const int base = warp == kScoreWarp ? 0 : plan.k_slots, slots = warp == kScoreWarp ? plan.k_slots : plan.v_slots;
            struct Place {
                int slot;
                uint32_t ph;
            };
            auto behind = [&](Place a) { return a.slot + 1 == base + slots ? Place{base, a.ph ^ 1} : Place{a.slot + 1, a.ph}; };
            // (threads and copies of the other block arrive at all of these barriers)
            auto ready = [&](Place a) { return mbar_test_cluster(smem_addr(&sh.kv_full[a.slot]), a.ph); };
            auto wait_both = [&](uint64_t *bar, uint32_t parity) { ok = __all_sync(~0u, ok && mbar_wait_cluster(smem_addr(bar), parity, status)); };
            Place at{base, 0};
            int tile = 0;
            // the next units, all there or the wait gave up
            auto arrived = [&](Place (&u)[kBatch], int count) {
                bool here = true;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    u[i] = at;
                    if (i < count) {
                        here &= ready(at);
                        at = behind(at);
                    }
                }
                if (__all_sync(~0u, here))
                    acquire_cluster();
                else
                    for (int i = 0; i < count && ok; ++i)
                        wait_both(&sh.kv_full[u[i].slot], u[i].ph);
                tc_fence_after();
                return ok;
            };
            PairWalk w(s, sh, units);
            if (warp == kScoreWarp) {
                constexpr uint32_t shape_s = mma_shape(kPairRows, kPairRows, false);
                int segment = 0;
                while (ok && __shfl_sync(~0u, (int)w.next(), 0)) {
                    const int n = __shfl_sync(~0u, w.t1 - w.t0, 0);
                    wait_both(&sh.q_full, segment++ & 1);
                    for (int j = 0; ok && j < n; ++j, ++tile) {  // S = Q K^T
                        if (tile > 1)
                            wait_both(&sh.p_full[tile & 1], (tile - 2) >> 1 & 1);  // S of two tiles before has been read
                        const uint32_t d = tm + 256 + (tile & 1) * 64;
                        for (int first = 0; ok && first < nk; first += kBatch * cw) {
                            const int count = min(kBatch, (nk - first + cw - 1) / cw);
                            Place u[kBatch];
                            if (!arrived(u, count))
                                break;
                            if (elect_one()) {
                                const uint64_t q = q_desc + (uint32_t)first * kQueryStep;
#pragma unroll
                                for (int i = 0; i < kBatch; ++i)
                                    if (i < count) {
                                        const uint64_t k = k_desc + (uint32_t)u[i].slot * unit_step;
#pragma unroll
                                        for (int ch = 0; ch < CW; ++ch)
                                            if (first + i * CW + ch < nk)
#pragma unroll
                                                for (int x = 0; x < 4; ++x)
                                                    mma_bf16_pair(d, q + (i * CW + ch) * kQueryStep + x * 2, k + ch * kChunkStep + x * 2, shape_s,
                                                                  i > 0 || ch > 0 || x > 0 || first > 0);
                                        mma_commit_pair(smem_addr(&sh.kv_empty[u[i].slot]));
                                    }
                                if (first + kBatch * cw >= nk) {
                                    mma_commit_pair(smem_addr(&sh.s_full[tile & 1]));
                                    if (j + 1 == n)
                                        mma_commit_pair(smem_addr(&sh.q_empty));
                                }
                            }
                            __syncwarp();
                        }
                    }
                }
            } else {
                const int v_units = 2 * ((plan.vch + cw - 1) / cw);
                while (ok && __shfl_sync(~0u, (int)w.next(), 0)) {
                    const int n = __shfl_sync(~0u, w.t1 - w.t0, 0);
                    for (int j = 0; ok && j < n; ++j, ++tile) {  // O (+)= P V
                        for (int first = 0; ok && first < v_units; first += kBatch) {
                            const int count = min(kBatch, v_units - first);
                            Place u[kBatch];
                            if (!arrived(u, count))
                                break;
                            if (first == 0) {
                                wait_both(&sh.p_full[tile & 1], tile >> 1 & 1);
                                if (!ok)
                                    break;
                                tc_fence_after();
                            }
                            if (elect_one()) {
                                const uint64_t pa = p_desc + (uint32_t)((tile & 1) * 2) * kQueryStep;
#pragma unroll
                                for (int i = 0; i < kBatch; ++i)
                                    if (i < count) {
                                        const int half = (first + i) & 1, to = (first + i) / 2 * cw * 64;
                                        const uint32_t shape = mma_shape(kPairRows, 2 * min(cw * 64, v_half - to), true);
                                        const uint64_t v = v_desc + (uint32_t)u[i].slot * unit_step;
#pragma unroll
                                        for (int k = 0; k < 4; ++k)
                                            mma_bf16_pair(tm + to, pa + half * kQueryStep + k * 2, v + k * sixteen, shape, half > 0 || k > 0 || j > 0);
                                        mma_commit_pair(smem_addr(&sh.kv_empty[u[i].slot]));
                                    }
                                if (first + kBatch >= v_units)
                                    mma_commit_pair(smem_addr(&sh.pv_done[tile & 1]));
                            }
                            __syncwarp();
                        }
                    }
                }
            }
            // nothing may be in flight when the blocks free their memory, a wait that gave up included
            if (elect_one())
                mma_commit_pair(smem_addr(&sh.drained));
            __syncwarp();
            mbar_wait(smem_addr(&sh.drained), 0, status);
            __syncwarp();
        }
    } else if (warp < kQueryWarp) {
        // ------------------------------------------------ rows by TMA, counted on the even block's barriers
        // (two warps for K, two for V, each with slots of its own: one took some 450 cycles a unit, with eight units a tile of 2048 cycles)
        const bool values = warp >= kCopyWarp + kCopyWarps / 2;
        const int base = values ? plan.k_slots : 0, slots = values ? plan.v_slots : plan.k_slots;
        const uint32_t kv_smem = smem_addr(kv_mem), full0 = at_rank(smem_addr(&sh.kv_full[0]), 0);
        const bool image = s.image_rows > 0;
        const int none = (int)(image ? (int64_t)s.n_groups * s.image_rows / 8 : p.n_pages * p.page_size / 8);  // a group past the end reads as zeros
        const int copies = 8 / plan.box_groups;
        int slot = base, filled = 0, last_filled = -1;
        uint32_t ph = 0;
        const int filler = (warp - kCopyWarp) % 2;
        PairWalk w(s, sh, units);
        while (ok && w.next()) {
            const int32_t *table = p.block_table + (int64_t)w.q.first * p.table_stride;
            // lane % 16 has one of a tile's groups of eight rows
            auto look_up = [&](int t) {
                const int row = t * kPairRows + (lane & 15) * 8;
                if (t >= w.t1)
                    return none;
                if (image)
                    return (w.g * s.image_rows + row) >> 3;
                if (row >= w.q.shared)
                    return none;
                return __ldg(table + p.by_page.quotient(row)) * (p.page_size / 8) + ((int)p.by_page.remainder(row) >> 3);
            };
            // 64 rows from group `first` of the tile on, chunks from `chunk` on
            auto fill = [&](int at, bool whole, int first, int chunk) {
                if (ring_filler(slot - base) == filler && ok) {
                    const int g = __shfl_sync(~0u, at, first + (whole ? lane * plan.box_groups : lane) % 8);
                    if (filled >= slots) {
                        ok = mbar_wait(smem_addr(&sh.kv_empty[slot]), ph ^ 1, status);
                        ok = __all_sync(~0u, ok);
                    }
                    if (ok) {
                        if (rank == 0 && lane == 0)
                            mbar_arrive_expect_tx(smem_addr(&sh.kv_full[slot]), 2 * unit_bytes);
                        if (lane < (whole ? copies : 8))
                            tma_load_4d_pair(kv_smem + slot * unit_bytes + lane * (whole ? plan.box_groups : 1) * group_bytes, whole ? &boxes : &groups,
                                             0, 0, chunk, g, full0 + slot * 8);
                        __syncwarp();
                        last_filled = filled;
                    }
                }
                ++filled;
                if (++slot == base + slots) {
                    slot = base;
                    ph ^= 1;
                }
            };
            int now = look_up(w.t0);
            for (int t = w.t0; ok && t < w.t1; ++t) {
                const bool whole = image || (t + 1) * kPairRows <= w.q.shared;
                const int next = look_up(t + 1);
                if (values)
                    for (int at = 0; at < plan.vch; at += cw) {
                        fill(now, whole, 0, rank * plan.vch + at);
                        fill(now, whole, 8, rank * plan.vch + at);
                    }
                else
                    for (int first = 0; first < nk; first += cw)
                        fill(now, whole, rank * 8, first);
                now = next;
            }
        }
        // no copy outlives the blocks, after a wait that gave up either (the even block's barriers count both blocks' copies)
        if (rank == 0 && lane == 0 && !ok)
            for (int k = last_filled; k >= 0 && k > last_filled - slots; --k)
                if (ring_filler(k % slots) == filler)
                    mbar_wait(smem_addr(&sh.kv_full[base + k % slots]), (k / slots) & 1, status);
        __syncwarp();
    } else {
        // ------------------------------------------------ queries, by copies of sixteen bytes
        const int qt = tid - 32 * kQueryWarp, unit = qt & 7;
        const uint32_t q_full = at_rank(smem_addr(&sh.q_full), 0);
        int segment = 0;
        PairWalk w(s, sh, units);
        while (ok && w.next()) {
            if (segment > 0) {
                ok = mbar_wait(smem_addr(&sh.q_empty), (segment - 1) & 1, status);
                ok = __all_sync(~0u, ok);
                if (!ok)
                    break;
            }
            ++segment;
            const int first = w.item() * kPairRows + rank * kHalf, rows = w.q.rows - first;
            for (int row = qt >> 3; row < kHalf; row += 4 * kQueryWarps) {
                // (rows past the item's end are zeros)
                const uint32_t flat = (uint32_t)(w.q.row0 + first + (row < rows ? row : 0)), token = p.by_heads.quotient(flat);
                const uint8_t *src = static_cast<const uint8_t *>(p.q) + unit * 16;
                if (row < rows)
                    src += ((int64_t)token * p.q_token_stride + (int64_t)(flat - token * (uint32_t)p.n_heads) * p.q_head_stride) * 2;
                const uint32_t dst = smem_addr(q_mem) + row * 128 + ((unit ^ (row & 7)) << 4);
#pragma unroll 4
                for (int ch = 0; ch < nk; ++ch)
                    copy_async_16(dst + ch * kQueryChunk, src + ch * 128, row < rows);
            }
            copy_async_wait();
            fence_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_cluster(q_full);
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_barrier();  // nothing of the other block's is under way to this one, and the pair's products are done
    if (warp == kScoreWarp) {
        mbar_wait(smem_addr(&sh.drained), 0, status);  // (the odd block: the last arrivals from the other one)
        tc_fence_after();
        tmem_free_pair(tmem, 512);
    }
}

// One block a group: how many rows the prefix part takes, and for the group's requests where their own rows begin.
__global__ void __launch_bounds__(256) shared_plan_kernel(const AttnParams p, const int32_t *__restrict__ cu_groups,
                                                         const int32_t *__restrict__ shared_rows, int least, const SharedPlan s)
{
    pdl_wait();
    pdl_trigger();
    __shared__ int fewest, reader;  // reader: the first request with new tokens, whose table is read
    const int g = blockIdx.x, tid = threadIdx.x;
    auto bound = [&](int i) { return min(max(__ldg(cu_groups + i), 0), p.n_req); };
    const int r0 = bound(g), r1 = max(bound(g + 1), r0);
    auto token = [&](int r) { return (int)min((int64_t)max(__ldg(p.cu_q + r), 0), p.n_tokens); };
    int most = min(max(__ldg(shared_rows + g), 0), p.width * p.page_size);
    if (s.image_rows > 0)
        most = min(most, s.image_rows);
    if (tid == 0) {
        fewest = most;
        reader = r1;
    }
    __syncthreads();
    // Rows that every new token sees: the first one of each request sees the fewest.  (None where a request has more rows than
    // its table lists, so that the rows behind a prefix end with the table.)
    for (int r = r0 + tid; r < r1; r += 256) {
        const int at = __ldg(p.cu_q + r), end = __ldg(p.cu_q + r + 1);
        if (min((int64_t)end, p.n_tokens) > max(at, 0)) {
            atomicMin(&reader, r);
            const int held = __ldg(p.seq_lens + r) - (end - at) + 1;
            const int all = max(__ldg(p.seq_lens + r), 0);
            const bool listed = (int)p.by_ratio.quotient((uint32_t)all) <= p.width * p.page_size;
            atomicMin(&fewest, held <= 0 || !listed ? 0 : (int)p.by_ratio.quotient((uint32_t)held));
        }
    }
    __syncthreads();
    const int pages = reader < r1 ? (int)p.by_page.quotient((uint32_t)fewest) : 0, first = reader;
    __syncthreads();
    if (tid == 0)
        fewest = pages;
    __syncthreads();
    // pages that lie in the cache, up to the first that does not
    for (int i = tid; i < pages; i += 256) {
        const int page = __ldg(p.block_table + (int64_t)first * p.table_stride + i);
        if (page < 0 || page >= p.n_pages)
            atomicMin(&fewest, i);
    }
    __syncthreads();
    const int row0 = token(r0) * p.n_heads, rows = max(token(r1) * p.n_heads - row0, 0);
    int shared = fewest * p.page_size;
    if (shared < least || r1 - r0 < 2 || rows == 0)
        shared = 0;
    if (tid == 0)
        s.groups[g] = GroupInfo{shared, (shared + kPairRows - 1) / kPairRows, row0, rows, first, shared ? (rows + kPairRows - 1) / kPairRows : 0};
    for (int r = r0 + tid; r < r1; r += 256)
        s.own[r] = make_int2(shared, g);
    // requests outside of all groups
    if (g == 0)
        for (int r = tid; r < r0; r += 256)
            s.own[r] = make_int2(0, -1);
    if (g + 1 == s.n_groups)
        for (int r = bound(g + 1) + tid; r < p.n_req; r += 256)
            s.own[r] = make_int2(0, -1);
}

// The prefixes' rows as bf16 rows of whole tiles, a warp a row; zeros past a prefix's end.  Blocks (x, group).
__global__ void __launch_bounds__(256) shared_image_kernel(const AttnParams p, const SharedPlan s)
{
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, g = blockIdx.y;
    const bool bits8 = p.cache_dtype == CSA_DTYPE_E4M3;
    const GroupInfo q = s.groups[g];
    for (int row = blockIdx.x * 8 + (threadIdx.x >> 5); row < q.tiles * kPairRows; row += gridDim.x * 8) {
        const int64_t to = (int64_t)g * s.image_rows + row;
        int64_t slot = -1;
        if (row < q.shared)
            slot = (int64_t)__ldg(p.block_table + (int64_t)q.first * p.table_stride + p.by_page.quotient(row)) * p.page_size +
                   p.by_page.remainder(row);
        uint16_t *dst = s.image + to * p.head_dim;
        for (int col = lane * 8; col < p.head_dim; col += 256) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (slot >= 0) {
                if (bits8) {
                    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(p.cache) + slot * p.cache_stride + col));
                    auto two = [](uint32_t e) {
                        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)e, __NV_E4M3);
                        return f2_to_bf16x2(__half22float2(*reinterpret_cast<const __half2 *>(&h)));
                    };
                    v = make_uint4(two(w.x & 0xffffu), two(w.x >> 16), two(w.y & 0xffffu), two(w.y >> 16));
                } else {
                    v = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.cache) + slot * p.cache_stride + col));
                }
            }
            *reinterpret_cast<uint4 *>(dst + col) = v;
        }
        if (bits8 && lane == 0)
            s.image_scales[to] = slot >= 0 ? __ldg(p.row_scales + slot) : 0.0f;
    }
}

// Joins the parts of the items' own rows and of their prefixes, in order.  Bound by a chain of five dependent reads, so where there
// are many rows a warp has two of them, whole (128 requests' 8192 rows: 30.3 us with a warp for 128 columns of one row, 23.6 so, from cold caches), and
// where there are few, whose parts may be many, 128 columns of one.
struct JoinRow {
    int64_t prefix, own;  // rows of the prefix's parts and of its own ones
    int n_prefix, n;
    float ref, inv;
};

template <bool MANY> __global__ void __launch_bounds__(256) shared_join_kernel(const AttnParams p, const SharedPlan s)
{
    pdl_wait();
    pdl_trigger();
    constexpr int kRows = MANY ? 2 : 1, kLanes = 32 / kRows;  // rows of a warp; lanes that look a row's sums up
    const int lane = threadIdx.x & 31, unit = blockIdx.y * 8 + (threadIdx.x >> 5), stripes = p.v_dim / 128;
    const int row0 = MANY ? unit * kRows : unit / stripes;
    if ((int)blockIdx.x >= *s.n_items)
        return;
    const OwnItem item = s.items[blockIdx.x];
    if (row0 >= item.rows)
        return;
    const int row = min(row0 + lane / kLanes, item.rows - 1), flat = item.row + row;
    JoinRow mine;
    const RowParts prefix = parts_of(s, item.group, flat);
    mine.prefix = (int64_t)prefix.first * kPairRows + prefix.row;
    mine.own = (int64_t)item.slot * kOwnRows + row;
    mine.n_prefix = prefix.n;
    mine.n = prefix.n + item.parts;
    auto sums = [&](const JoinRow &r, int k) {
        return __ldcg(k < r.n_prefix ? s.part_ml + r.prefix + (int64_t)k * kPairRows : s.own_ml + r.own + (int64_t)(k - r.n_prefix) * kOwnRows);
    };
    const float sink = p.sink ? __ldg(p.sink + p.by_heads.remainder((uint32_t)flat)) * kLog2E : -INFINITY;
    float top = sink;
    float2 kept = make_float2(-INFINITY, 0.0f);
    for (int k = lane % kLanes; k < mine.n; k += kLanes) {
        kept = sums(mine, k);
        top = fmaxf(top, kept.x);
    }
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    mine.ref = top == -INFINITY ? 0.0f : top;
    // (the sums of up to sixteen parts are still there)
    float tot = 0.0f;
    for (int k = lane % kLanes; k < mine.n; k += kLanes) {
        const float2 ml = mine.n <= kLanes ? kept : sums(mine, k);
        tot = fmaf(part_weight(ml.x, mine.ref), ml.y, tot);
    }
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1)
        tot += __shfl_xor_sync(~0u, tot, o);
    tot += exp2_fast(sink - mine.ref);
    mine.inv = tot == 0.0f ? 0.0f : 1.0f / tot;
    if (p.lse && lane % kLanes == 0 && row == row0 + lane / kLanes && (MANY || unit % stripes == 0))
        p.lse[flat] = tot == 0.0f ? -INFINITY : (mine.ref + log2f(tot)) * kLn2;

    constexpr int kStripes = MANY ? 4 : 1;
#pragma unroll
    for (int h = 0; h < kRows; ++h) {
        if (row0 + h >= item.rows)
            break;
        JoinRow r;
        r.prefix = __shfl_sync(~0u, mine.prefix, h * kLanes);
        r.own = __shfl_sync(~0u, mine.own, h * kLanes);
        r.n_prefix = __shfl_sync(~0u, mine.n_prefix, h * kLanes);
        r.n = __shfl_sync(~0u, mine.n, h * kLanes);
        r.ref = __shfl_sync(~0u, mine.ref, h * kLanes);
        r.inv = __shfl_sync(~0u, mine.inv, h * kLanes);
        const int col = (MANY ? 0 : unit % stripes) * 128 + lane * 4;
        const float *prefix_o = s.part_o + r.prefix * p.v_dim + col, *own_o = s.own_o + r.own * p.v_dim + col;
        float4 o[kStripes] = {};
#pragma unroll(MANY ? 3 : 8)
        for (int k = 0; k < r.n; ++k) {
            const float w = part_weight(sums(r, k).x, r.ref);
            const float *src = k < r.n_prefix ? prefix_o + (int64_t)k * kPairRows * p.v_dim : own_o + (int64_t)(k - r.n_prefix) * kOwnRows * p.v_dim;
#pragma unroll
            for (int i = 0; i < kStripes; ++i)
                if (!MANY || i < stripes) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(src + i * 128));
                    o[i] = make_float4(fmaf(w, v.x, o[i].x), fmaf(w, v.y, o[i].y), fmaf(w, v.z, o[i].z), fmaf(w, v.w, o[i].w));
                }
        }
        uint16_t *dst = static_cast<uint16_t *>(p.out) + (int64_t)(item.row + row0 + h) * p.v_dim + col;
#pragma unroll
        for (int i = 0; i < kStripes; ++i)
            if (!MANY || i < stripes)
                *reinterpret_cast<uint2 *>(dst + i * 128) = make_uint2(f2_to_bf16x2(make_float2(o[i].x * r.inv, o[i].y * r.inv)),
                                                                       f2_to_bf16x2(make_float2(o[i].z * r.inv, o[i].w * r.inv)));
    }
}

PairPlan make_plan(const AttnParams &p)
{
    PairPlan m{};
    m.nk = p.head_dim / 64;
    m.vch = p.v_dim / 128;
    m.cw = m.vch < 2 ? m.vch : 2;
    const size_t unit = (size_t)m.cw * 8 * 1024, fixed = (size_t)(m.nk + 4) * kQueryChunk + 1024;
    const size_t limit = 227 * 1024 - sizeof(PairShared);
    // the rings' sizes go as the units of a tile, and are two or more: an MMA warp waits for two units at once
    const int fit = (int)((limit - fixed) / unit), slots = fit > kMaxSlots ? kMaxSlots : fit;
    const PairRings rings = pair_rings(slots, (m.nk + m.cw - 1) / m.cw, 2 * ((m.vch + m.cw - 1) / m.cw), kBatch);
    m.k_slots = rings.k;
    m.v_slots = rings.v;
    m.smem = fixed + slots * unit;
    // a block an SM, beside none of the attention by requests (90 KB or more), which has tensor memory too
    m.smem = m.smem < 140 * 1024 ? 140 * 1024 : m.smem;
    const int groups = needs_image(prefix_call(p, 0)) ? 8 : p.page_size / 8;
    for (m.box_groups = 8; groups % m.box_groups; m.box_groups /= 2) {}
    return m;
}

template <bool BITS8, int CW>
cudaError_t launch_pair(const AttnParams &p, const SharedPlan &s, const PairPlan &m, unsigned *status, cudaStream_t st)
{
    auto kern = latent_pair_kernel<BITS8, CW>;
    cudaError_t e = allow_max_smem(reinterpret_cast<const void *>(kern));
    CUtensorMap boxes = {}, groups = {};
    const bool image = s.image_rows > 0;
    const void *rows = image ? static_cast<const void *>(s.image) : p.cache;
    const int64_t n = image ? (int64_t)s.n_groups * s.image_rows : p.n_pages * p.page_size, stride = image ? p.head_dim : p.cache_stride;
    if (e == cudaSuccess)
        e = make_tensor_map_groups(&groups, rows, n, m.nk, stride, 1, m.cw);
    if (e == cudaSuccess)
        e = make_tensor_map_groups(&boxes, rows, n, m.nk, stride, m.box_groups, m.cw);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2] = {pdl_attribute(), {}};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cfg.stream = st;
    cfg.gridDim = dim3(2 * s.clusters);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = m.smem;
    return cudaLaunchKernelEx(&cfg, kern, p, s, m, boxes, groups, status);
}

template <bool BITS8>
cudaError_t launch_pair(const AttnParams &p, const SharedPlan &s, const PairPlan &m, unsigned *status, cudaStream_t st)
{
    return m.cw == 1 ? launch_pair<BITS8, 1>(p, s, m, status, st) : launch_pair<BITS8, 2>(p, s, m, status, st);
}

cudaError_t clusters_of(const AttnParams &p, const PairPlan &m, int *clusters)
{
    const void *fn = p.cache_dtype == CSA_DTYPE_E4M3 ? reinterpret_cast<const void *>(latent_pair_kernel<true, 2>)
                                                     : reinterpret_cast<const void *>(latent_pair_kernel<false, 2>);
    int resident = 0;
    const cudaError_t e = resident_blocks(fn, kThreads, m.smem, 2, &resident);
    *clusters = resident / 2;
    return e == cudaSuccess && *clusters < 1 ? cudaErrorInvalidConfiguration : e;
}

// Takes pieces of a workspace.
struct Pieces {
    uint8_t *base;
    size_t used;
    template <typename T> T *take(size_t n)
    {
        T *at = base ? reinterpret_cast<T *>(base + used) : nullptr;
        used += (n * sizeof(T) + 255) / 256 * 256;
        return at;
    }
};

}  // namespace

cudaError_t launch_shared_mma(const AttnParams &p, const int32_t *cu_groups, const int32_t *shared_rows, int n_groups, int num_sms,
                              cudaMemPool_t pool, unsigned *status, cudaStream_t st)
{
    const PairPlan m = make_plan(p);
    const PrefixCall call = prefix_call(p, n_groups);
    SharedPlan s{};
    cudaError_t e = clusters_of(p, m, &s.clusters);
    if (e != cudaSuccess)
        return e;
    s.n_groups = n_groups;
    s.max_items = (int)(p.n_tokens * p.n_heads / kPairRows) + n_groups;
    s.image_rows = image_rows(call);
    s.max_own = (int)own_items(call);
    const size_t slots = (size_t)s.max_items + s.clusters;
    const size_t own_slots = latent_behind_slots(p, num_sms);
    auto lay_out = [&](void *at) {
        Pieces w{static_cast<uint8_t *>(at), 0};
        s.own = w.take<int2>(p.n_req);
        s.groups = w.take<GroupInfo>(n_groups);
        s.sums = w.take<GroupSums>(n_groups);
        s.total = w.take<long long>(1);
        s.image = w.take<uint16_t>((size_t)n_groups * s.image_rows * p.head_dim);
        s.image_scales = w.take<float>(p.cache_dtype == CSA_DTYPE_E4M3 ? (size_t)n_groups * s.image_rows : 0);
        s.part_o = w.take<float>(slots * kPairRows * p.v_dim);
        s.part_ml = w.take<float2>(slots * kPairRows);
        s.items = w.take<OwnItem>(s.max_own);
        s.n_items = w.take<int>(1);
        s.own_o = w.take<float>(own_slots * kOwnRows * p.v_dim);
        s.own_ml = w.take<float2>(own_slots * kOwnRows);
        return w.used;
    };
    void *workspace = nullptr;
    e = cudaMallocFromPoolAsync(&workspace, lay_out(nullptr), pool, st);
    if (e != cudaSuccess)
        return e;
    lay_out(workspace);

    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = st;
    cfg.blockDim = dim3(256);
    cfg.gridDim = dim3(n_groups);
    e = cudaLaunchKernelEx(&cfg, shared_plan_kernel, p, cu_groups, shared_rows, kPairRows, (const SharedPlan)s);
    if (e == cudaSuccess && s.image_rows > 0) {
        const int most = (s.image_rows + 7) / 8, each = (8 * num_sms + n_groups - 1) / n_groups;
        cfg.gridDim = dim3(most < each ? most : each, n_groups);
        e = cudaLaunchKernelEx(&cfg, shared_image_kernel, p, (const SharedPlan)s);
    }
    if (e == cudaSuccess)
        e = p.cache_dtype == CSA_DTYPE_E4M3 ? launch_pair<true>(p, s, m, status, st) : launch_pair<false>(p, s, m, status, st);
    if (e == cudaSuccess)
        e = launch_latent_behind(p, s, num_sms, status, st);
    if (e == cudaSuccess) {
        const bool many = s.max_own > num_sms;
        cfg.gridDim = dim3(s.max_own, many ? kOwnRows / 16 : kOwnRows * (p.v_dim / 128) / 8);
        e = cudaLaunchKernelEx(&cfg, many ? shared_join_kernel<true> : shared_join_kernel<false>, p, (const SharedPlan)s);
    }
    const cudaError_t e2 = cudaFreeAsync(workspace, st);
    return e == cudaSuccess ? e2 : e;
}

}  // namespace csa
