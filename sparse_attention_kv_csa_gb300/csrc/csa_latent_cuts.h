// How the attention's work is divided: whole-number arithmetic that the kernel and, compiled for the host, its tests run.
#pragma once

#include <stdint.h>

#include <algorithm>

#ifdef __CUDACC__
#define CSA_BOTH __host__ __device__ __forceinline__
#else
#define CSA_BOTH inline
#endif

namespace csa {

#ifndef __CUDA_ARCH__
using std::max;
using std::min;
#endif

// n / d for 0 <= n < 2^31 by a multiplication (T. Granlund and P. Montgomery, "Division by invariant integers using
// multiplication", PLDI 1994): with l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1, n / d = (hi(m n) + n) >> l.
struct Divider {
    uint32_t m, l, d;
    Divider() = default;
    explicit Divider(uint32_t divisor) : m(0), l(0), d(divisor)
    {
        while (l < 31 && (1u << l) < d)
            ++l;
        m = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << l) - d)) / d + 1);
    }
    CSA_BOTH uint32_t quotient(uint32_t n) const
    {
#ifdef __CUDA_ARCH__
        return (__umulhi(m, n) + n) >> l;
#else
        return ((uint32_t)((uint64_t)m * n >> 32) + n) >> l;
#endif
    }
    CSA_BOTH uint32_t remainder(uint32_t n) const { return n - quotient(n) * d; }
};

// Units of an item besides its tiles, for its queries and output: a decode step of 64 requests 83.8, 81.2 and 80.2 us with
// 1, 2 and 3, of 129 requests with 8-bit rows 150.2, 148.0 and 145.4.
constexpr int kHead = 3;
// Units of a block's share at least.  Eight requests of 1024 rows: 26.1, 23.5 and 22.2 us with 4, 3 and 2; one of 16384
// rows: 26.9, 27.6 and 32.0.
constexpr int kMinUnits = 3;

// The same for an item of a shared prefix.
constexpr int kPairHead = 2;

// How many blocks share the units.
CSA_BOTH int sharing(long long total, int blocks) { return (int)max(1ll, min(total / kMinUnits, (long long)blocks)); }

// Block c's first unit, of g blocks.
CSA_BOTH long long cut(long long total, int c, int g)
{
    return total < (1 << 20) ? (long long)((uint32_t)total * (uint32_t)c / (uint32_t)g) : total * c / g;  // c < 4096
}

// The block whose share holds a unit.
CSA_BOTH int holder(long long unit, long long total, int g)
{
    return total < (1 << 20) ? (int)(((uint32_t)(unit + 1) * (uint32_t)g - 1) / (uint32_t)total) : (int)(((unit + 1) * g - 1) / total);
}

// The rings of a shared prefix's K and V, in units: shares of `slots` that go as the units of a tile, `least` each at least.
struct PairRings {
    int k, v;
};

CSA_BOTH PairRings pair_rings(int slots, int k_units, int v_units, int least)
{
    const int k = (slots * k_units + (k_units + v_units) / 2) / (k_units + v_units);
    PairRings r;
    r.k = k < least ? least : k > slots - least ? slots - least : k;
    r.v = slots - r.k;
    return r;
}

// Which of the two warps that fill a ring has a slot: always the same one, whether the ring has an even or an odd number of them.  A
// barrier's parity tells a phase that is over from one that has not begun only to who took the one before.
CSA_BOTH int ring_filler(int slot) { return slot & 1; }

// What the choice of a way through a call with shared prefixes goes by: all of it is known to the host.
struct PrefixCall {
    long long n_tokens;
    int n_heads, n_req, n_groups, head_dim, v_dim;
    bool bits8;
    long long n_pages;
    int page_size, width;
};

constexpr int kPairRows = 128;  // query rows of an item of a shared prefix, and cache rows of its tiles
constexpr int kOwnRows = 64;    // query rows of an item of the rows behind it

// Widths that the attentions' tensor-core kernels take.
CSA_BOTH bool on_tensor_cores(int head_dim, int v_dim) { return head_dim % 64 == 0 && head_dim <= 576 && v_dim % 64 == 0 && v_dim <= 512; }

// The most items of rows behind prefixes.
CSA_BOTH long long own_items(const PrefixCall &c) { return c.n_tokens * c.n_heads / kOwnRows + c.n_req; }

// Rows that TMA does not bring as bf16 in whole groups of eight are copied once into an image of the prefix.
CSA_BOTH bool needs_image(const PrefixCall &c) { return c.bits8 || c.page_size % 8 != 0; }

// Rows of a group's image: as many as a table lists and the cache has (a table may have room for far more), within a GiB for all groups.
// Rows of a prefix past them are read by request.
CSA_BOTH int image_rows(const PrefixCall &c)
{
    if (!needs_image(c))
        return 0;
    const long long room = (1ll << 30) / ((long long)c.n_groups * c.head_dim * 2) / kPairRows * kPairRows;
    const long long pages = min((long long)c.width, c.n_pages);
    return (int)min(room, (pages * c.page_size + kPairRows - 1) / kPairRows * kPairRows);
}

// Whether prefixes are read apart.  By requests an SM does a tile of 64 query rows x 64 rows in some 1 us, here the prefix's in 0.6, behind
// some 25 us of launches, parts and their join.  Measured, in such tiles an SM by the table's width: 24 of 576 columns 59.5 us
// here, 54.8 by requests; another 24 45.8 and 49.6; 30 of 256 columns 38.5 and 39.6; of 128 and 192 columns, two blocks an SM by
// requests, 24: 43.5 and 35.4, 39: 55.3 and 49.7, 54: 54.1 and 41.1, 58: 36.8 and 50.8, 103: 64.5 and 100.2, 275: 128.1 and 117.6; with
// four requests a group 48: 64.5 and 50.3; with an image 31: 77.9 and 54.0, 70: 121 and 123.  So the rule is a rough one (the two at
// 58 and 275 go the other way), and a table wider than its requests need counts as if it were full.
CSA_BOTH bool prefix_apart(const PrefixCall &c, int num_sms)
{
    if (!on_tensor_cores(c.head_dim, c.v_dim) || c.v_dim % 128 != 0 || c.n_groups < 1 || c.n_req < 2 ||
        (long long)c.width * c.page_size < kPairRows || (needs_image(c) && image_rows(c) < kPairRows))
        return false;
    const long long rows = c.n_tokens * c.n_heads / kOwnRows, items = max(rows, (long long)c.n_req);
    const long long tiles = ((long long)c.width * c.page_size + 63) / 64;
    if (items * tiles < (needs_image(c) || c.head_dim <= 192 || c.n_req < 8 * c.n_groups ? 64 : 24) * (long long)num_sms)
        return false;
    // (the parts of a prompt's many tokens would take too much room: they fill the machine request by request)
    return ((c.n_tokens * c.n_heads / kPairRows + c.n_groups) * kPairRows + own_items(c) * kOwnRows) * c.v_dim * 4 <= 1ll << 32;
}

// What a block does of an item of nt tiles, from its unit `off` on with `left` units to do: `take` units, of them tiles
// [t0, t1).  some: the item falls to this block too, by a tile or, without tiles, by its first unit.
struct Segment {
    int take, t0, t1;
    bool some;
};

CSA_BOTH Segment segment_of(int nt, int off, long long left, int head = kHead)
{
    Segment s;
    s.take = (int)min((long long)(nt + head - off), left);
    s.t0 = max(off - head, 0);
    s.t1 = max(off + s.take - head, 0);
    s.some = s.t1 > s.t0 || (nt == 0 && off == 0);
    return s;
}

}  // namespace csa
