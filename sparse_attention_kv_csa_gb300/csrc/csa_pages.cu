// Block tables, row offsets and slots of a paged cache of compressed rows, from the requests' lengths.
//
//   old_r = floor(before_r / ratio), new_r = max(floor(after_r / ratio), old_r)      rows before and after
//   held_r = ceil(old_r / page),     need_r = ceil(new_r / page)                     pages before and after
//   cu_rows = prefix sum of new - old,  cu_pages = prefix sum of need - held
//   table_out[r, c] = table[r, c] for c < held_r, free[taken + cu_pages_r + c - held_r] for c < need_r, else -1
//   slot of new row i of request r: table_out[r, row / page] * page + row % page with row = old_r + i
//
// Bound by launch latency for a decode step (a few hundred KB at most) and by the table's bytes for large batches.
// One launch: the prefix sums run over two integers a request, so every block forms all of them in shared memory
// (14000 requests are 112 KB) instead of waiting for another kernel, then takes its share of the table and slots.
#include "csa_device.cuh"
#include "csa_launch.h"
#include "csa_serving_launch.h"

namespace csa {
namespace {

constexpr int kThreads = 512;

struct Req {
    int old_rows, new_rows, held, need;
};

__device__ __forceinline__ Req request(const PageParams &p, int r)
{
    Req q;
    q.old_rows = max(__ldg(p.before + r), 0) / p.ratio;
    q.new_rows = max(max(__ldg(p.after + r), 0) / p.ratio, q.old_rows);
    q.held = q.old_rows / p.page_size + (q.old_rows % p.page_size != 0);
    q.need = q.new_rows / p.page_size + (q.new_rows % p.page_size != 0);
    return q;
}

// a + b of two counts, held at 2^31 - 1: in any order the same, and no offset formed of such sums goes astray.
__device__ __forceinline__ int sum(int a, int b) { return (int)min((unsigned)a + (unsigned)b, 0x7fffffffu); }

__global__ void __launch_bounds__(kThreads) page_tables_kernel(const PageParams p)
{
    extern __shared__ int sums[];
    int *cu_rows = sums, *cu_pages = sums + p.n_req + 1;
    __shared__ int part[2][kThreads / 32];
    __shared__ int widest;
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = p.n_req;
    if (tid == 0)
        widest = 0;
    __syncthreads();
    // Exclusive prefix sums: a thread adds up a stretch of requests, the threads' sums are scanned, the thread goes over
    // its stretch again.
    const int per = (n + kThreads - 1) / kThreads, lo = min(n, tid * per), hi = min(n, lo + per);
    int rows = 0, pages = 0, wide = 0;
#pragma unroll 4
    for (int r = lo; r < hi; ++r) {
        const Req q = request(p, r);
        rows = sum(rows, q.new_rows - q.old_rows);
        pages = sum(pages, q.need - q.held);
        wide = max(wide, q.need);
    }
    int a = rows, b = pages;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int ua = __shfl_up_sync(~0u, a, o), ub = __shfl_up_sync(~0u, b, o);
        if (lane >= o) {
            a = sum(a, ua);
            b = sum(b, ub);
        }
    }
    if (lane == 31) {
        part[0][warp] = a;
        part[1][warp] = b;
    }
    __syncthreads();
    int base_rows = 0, base_pages = 0;
    a = __shfl_up_sync(~0u, a, 1);
    b = __shfl_up_sync(~0u, b, 1);
    if (lane == 0)
        a = b = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
        const int pa = part[0][i], pb = part[1][i];
        if (i < warp) {
            a = sum(a, pa);
            b = sum(b, pb);
        }
        base_rows = sum(base_rows, pa);
        base_pages = sum(base_pages, pb);
    }
    for (int r = lo; r < hi; ++r) {
        const Req q = request(p, r);
        cu_rows[r] = a;
        cu_pages[r] = b;
        a = sum(a, q.new_rows - q.old_rows);
        b = sum(b, q.need - q.held);
    }
    if (tid == 0) {
        cu_rows[n] = base_rows;
        cu_pages[n] = base_pages;
    }
    if (blockIdx.x == 0) {
        wide = __reduce_max_sync(~0u, wide);
        if (lane == 0)
            atomicMax(&widest, wide);
    }
    __syncthreads();
    const int64_t first_free = p.taken ? max(__ldg(p.taken), 0) : 0;
    auto fresh = [&](int64_t k) { return first_free + k < p.n_free ? __ldg(p.free_pages + first_free + k) : -1; };
    if (blockIdx.x == 0) {
        for (int r = tid; r <= n; r += kThreads)
            p.cu_rows[r] = cu_rows[r];
        if (tid == 0) {
            const int64_t left = max((int64_t)p.n_free - first_free, (int64_t)0);
            const int got = (int)min((int64_t)base_pages, left);
            p.counts[0] = base_rows;
            p.counts[1] = got;
            p.counts[2] = base_pages - got;
            p.counts[3] = widest;
        }
    }
    // table: one warp a stretch of a request's columns
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32), me = (int64_t)blockIdx.x * (kThreads / 32) + warp;
    const int chunks = (p.width + 511) / 512;
    for (int64_t u = me; u < (int64_t)n * chunks; u += warps) {
        const int r = (int)(u / chunks), c0 = (int)(u % chunks) * 512;
        const Req q = request(p, r);
        const int64_t add = (int64_t)cu_pages[r] - q.held;
        const int64_t in_row = (int64_t)r * p.table_stride, out_row = (int64_t)r * p.width;
        const int end = min(p.width, c0 + 512);
        for (int c = c0 + lane; c < end; c += 32 * 4) {
            int id[4];  // four loads under way
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int cu = c + 32 * u;
                id[u] = -1;
                if (cu < end) {
                    if (cu < q.held)
                        id[u] = p.table[in_row + cu];
                    else if (cu < q.need)
                        id[u] = fresh(add + cu);
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (c + 32 * u < end)
                    p.table_out[out_row + c + 32 * u] = id[u];
        }
    }
    // slots: the request of row i by bisection of the offsets in shared memory
    for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < p.capacity; i += (int64_t)gridDim.x * kThreads) {
        int64_t slot = -1;
        if (i < base_rows) {
            int lo = 0, hi = n;  // cu_rows[lo] <= i < cu_rows[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu_rows[mid] <= i)
                    lo = mid;
                else
                    hi = mid;
            }
            const Req q = request(p, lo);
            const int row = q.old_rows + (int)(i - cu_rows[lo]);
            const int c = row / p.page_size;
            if (c < p.width) {
                const int id = c < q.held ? p.table[(int64_t)lo * p.table_stride + c]
                                          : fresh((int64_t)cu_pages[lo] + c - q.held);
                if (id >= 0)
                    slot = (int64_t)id * p.page_size + row % p.page_size;
            }
        }
        p.slots[i] = slot;
    }
}

}  // namespace

cudaError_t launch_page_tables(const PageParams &p, int num_sms, cudaStream_t st)
{
    const size_t smem = 2 * ((size_t)p.n_req + 1) * sizeof(int);
    cudaError_t e = allow_max_smem(reinterpret_cast<const void *>(page_tables_kernel));
    if (e != cudaSuccess)
        return e;
    // a block for every 16 stretches of the table or 512 slots, at most one an SM
    const int64_t a = ((int64_t)p.n_req * ((p.width + 511) / 512) + 15) / 16, b = ((int64_t)p.capacity + kThreads - 1) / kThreads;
    int64_t grid = a > b ? a : b;
    grid = grid < 1 ? 1 : grid > num_sms ? num_sms : grid;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, page_tables_kernel, p);
}

}  // namespace csa
