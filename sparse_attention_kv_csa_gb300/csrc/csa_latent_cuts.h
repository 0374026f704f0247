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

#ifndef __CUDA_ARCH__
using std::max;
using std::min;
#endif

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

// What a block does of an item of nt tiles, from its unit `off` on with `left` units to do: `take` units, of them tiles
// [t0, t1).  some: the item falls to this block too, by a tile or, without tiles, by its first unit.
struct Segment {
    int take, t0, t1;
    bool some;
};

CSA_BOTH Segment segment_of(int nt, int off, long long left)
{
    Segment s;
    s.take = (int)min((long long)(nt + kHead - off), left);
    s.t0 = max(off - kHead, 0);
    s.t1 = max(off + s.take - kHead, 0);
    s.some = s.t1 > s.t0 || (nt == 0 && off == 0);
    return s;
}

}  // namespace csa
