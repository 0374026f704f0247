// The norm's ring (csa_norm_ring.cuh) on the host, over barriers and copies that only keep count: copy number `stuck` of a
// team's stages never lands, the others land at once or, the `late` ones after it, when they are first waited for.
#include <stdint.h>
#include <vector>

#define __device__
#define __forceinline__ inline

namespace {
struct Barrier {
    int issued = 0, landed = 0, waited = 0;  // phases begun by a fill, complete, waited for
    int fill = -1;                           // number of the last fill
};
Barrier g_bar[16];
int g_fills, g_stuck, g_faults, g_copies;
bool g_late;

uint32_t smem_addr(const void *p) { return (uint32_t)(reinterpret_cast<uintptr_t>(p) >> 3); }
Barrier &barrier(uint32_t a);
void mbar_init(uint32_t, int) {}
void mbar_init_fence() {}
void __syncthreads() {}
void land(Barrier &b)
{
    if (b.fill != g_stuck)
        b.landed = b.issued;
}
void mbar_arrive_expect_tx(uint32_t bar, uint32_t)
{
    Barrier &b = barrier(bar);
    g_faults += b.issued != b.landed;  // the phase before is still open
    ++b.issued;
    b.fill = g_fills++;
    if (!g_late || b.fill < g_stuck)
        land(b);
}
void bulk_g2s(uint32_t, const void *, uint32_t, uint32_t) { ++g_copies; }
bool mbar_wait(uint32_t bar, uint32_t parity, unsigned *status)
{
    Barrier &b = barrier(bar);
    land(b);
    if (b.issued > 0 && (uint32_t)((b.issued - 1) & 1) == parity)
        b.waited = b.issued;
    // the phase of this parity is over when another is under way
    const bool over = (uint32_t)(b.landed & 1) != parity;
    if (!over)
        *status = 1;
    return over;
}
}  // namespace

#include "csa_norm_ring.cuh"

static uint64_t g_full[16];
namespace {
Barrier &barrier(uint32_t a) { return g_bar[a - smem_addr(g_full)]; }
}  // namespace

// A team's first thread over n_rows rows, row 0 first, `step` apart.  Returns the faults: a fill of an open phase, a fill that
// is never waited for, a row read after a wait that gave up counted as good, or a timeout that is not recorded.
extern "C" int ring_faults(int stages, long long n_rows, long long step, int arrays, int stuck, int late, int *fills)
{
    using namespace csa;
    for (Barrier &b : g_bar)
        b = Barrier();
    g_fills = g_faults = g_copies = 0;
    g_stuck = stuck;
    g_late = late != 0;
    unsigned status = 0;
    alignas(16) static uint8_t mem[16];
    const Ring ring{mem, g_full, stages, 16, arrays, &status};
    const void *some = mem;
    auto refill = [&](int64_t row, int stage) {
        if (row < n_rows)
            ring.fill(stage, some, arrays > 1 ? some : nullptr, arrays > 2 ? some : nullptr);
    };
    RingAt at;
    ring.init(true);
    for (int i = 0; i < stages; ++i)
        refill(i * step, i);
    int64_t good = 0;
    for (int64_t row = 0; row < n_rows; row += step) {
        ring.wait(at, true, row, step, n_rows);
        good += at.ok;
        if (at.ok)
            refill(row + stages * step, at.stage);
        ring.next(at);
    }
    for (const Barrier &b : g_bar)
        g_faults += b.waited != b.issued;
    const int64_t rows = (n_rows + step - 1) / step;
    const bool hit = stuck >= 0 && stuck < rows;
    g_faults += good != (hit ? stuck : rows);
    g_faults += (status != 0) != hit;
    g_faults += g_copies != g_fills * arrays;
    *fills = g_fills;
    return g_faults;
}
