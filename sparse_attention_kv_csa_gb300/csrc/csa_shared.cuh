// What the attention over a shared prefix hands from one kernel to the next (csa_shared.cu has the whole).
#pragma once

#include <stdint.h>

#include "csa_latent_cuts.h"

#ifdef __CUDACC__
#include "csa_tcgen05.cuh"
#endif

namespace csa {

struct GroupInfo {
    int shared;  // rows that the group's prefix part takes: whole pages, seen by every new token of the group
    int tiles;
    int row0, rows;  // its query rows: (token, head) pairs
    int first;       // its first request with new tokens, whose table lists the prefix
    int items;
};

struct GroupSums {
    long long unit_base;
    int item_base, items;
};

// An item of 64 query rows of one request, and the parts of its own rows.
struct OwnItem {
    int row, rows;
    int group;        // whose prefix its rows see besides (-1: none)
    int parts, slot;  // slots slot, slot + 1, ...
};

struct SharedPlan {
    int n_groups, clusters;
    int max_items;
    int image_rows;       // rows of a group's image; 0: the prefix is read from the cache itself
    int2 *own;            // [n_req] of each request: rows that the prefix part takes, group (-1: none)
    GroupInfo *groups;    // [n_groups]
    GroupSums *sums;      // [n_groups]
    long long *total;     // units of all items
    uint16_t *image;      // [n_groups][image_rows][head_dim] bf16
    float *image_scales;  // [n_groups][image_rows], 8-bit rows only
    float *part_o;        // [max_items + clusters][128][v_dim]
    float2 *part_ml;      // [max_items + clusters][128]  (m, l)
    int max_own;          // own_items()
    OwnItem *items;       // [max_own]
    int *n_items;
    float *own_o;         // [max_own + blocks][64][v_dim]
    float2 *own_ml;       // [max_own + blocks][64]
};

#ifdef __CUDACC__
// What a part's sums count for beside a reference of m.
__device__ __forceinline__ float part_weight(float part_m, float m)
{
    return part_m == m ? 1.0f : exp2_fast(part_m - m);  // (-inf beside -inf too)
}

// The parts of a query row of group g: part k of n is row `row` of slot first + k.  (A part's slot is its item's number plus its
// cluster's: of the pairs (item, cluster) in the order of the units each has at least one of the two one higher than the one before.)
struct RowParts {
    int first, n, row;
};

__device__ __forceinline__ RowParts parts_of(const SharedPlan &s, int g, int flat_row)
{
    RowParts p{0, 0, 0};
    if (g < 0)
        return p;
    const GroupInfo info = s.groups[g];
    const GroupSums sums = s.sums[g];
    const int local = flat_row - info.row0, item = local / kPairRows;
    if (info.shared <= 0 || local < 0 || item >= sums.items)
        return p;
    const long long total = *s.total, unit = sums.unit_base + (long long)item * (info.tiles + kPairHead) + kPairHead;
    const int blocks = sharing(total, s.clusters), c0 = holder(unit, total, blocks);
    p.first = sums.item_base + item + c0;
    p.n = holder(unit + info.tiles - 1, total, blocks) - c0 + 1;
    p.row = local % kPairRows;
    return p;
}
#endif

}  // namespace csa
