// A team's ring of rows in shared memory: the arrays' rows side by side, refilled by the team's first thread once the
// team has read them.  Uses the barrier and copy primitives of csa_device.cuh, which is included before it.
#pragma once

#include <stdint.h>

namespace csa {
namespace {

constexpr int kMaxRing = 8;

// Where a thread stands in the ring.  ok: no wait of this thread has given up so far.
struct RingAt {
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
};

struct Ring {
    uint8_t *mem;
    uint64_t *full;
    int stages, row_bytes, arrays;
    unsigned *status;
    __device__ void init(bool first) const
    {
        if (first) {
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
    // Waits for the team's row (one of `step` apart, below n_rows).  A wait that gives up has set the status word (the
    // rows' results are then wrong, as documented) and is the thread's last; the first thread, which refills no stage from
    // then on, first waits out its copies under way, the given-up one among them, so that none outlives the block.
    __device__ void wait(RingAt &x, bool first, int64_t row, int64_t step, int64_t n_rows) const
    {
        if (!x.ok)
            return;
        x.ok = mbar_wait(smem_addr(full + x.stage), x.phase, status);
        if (!x.ok && first) {
            int stage = x.stage;
            uint32_t phase = x.phase;
            for (int i = 0; i < stages && row < n_rows; ++i, row += step) {
                mbar_wait(smem_addr(full + stage), phase, status);
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
    }
    __device__ void next(RingAt &x) const
    {
        if (++x.stage == stages) {
            x.stage = 0;
            x.phase ^= 1u;
        }
    }
};

}  // namespace
}  // namespace csa
