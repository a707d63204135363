// cache_tma.cuh -- tensor maps over the rows of a cache.
#pragma once

#include <cuda.h>

#include "cache_internal.cuh"

namespace qkr {

// Rows of one plane: the map's axes are (element, then row, head and page in
// the order of their strides).
struct PlaneMap {
    CUtensorMap m;
    int row_axis, head_axis;   // 1..3; the page has the third
    int box;                   // rows of one copy
};
struct CacheMaps {
    PlaneMap k, v;
};

// Maps of the K and V planes.  A copy is `box` rows, the largest of 16, 32, 64,
// 128 that divides the page and is at most `keys`; of bf16 rows 64 elements in
// the 128-byte swizzle, of 4-bit rows all code bytes (64-byte swizzle at D =
// 128, none at 64).
cudaError_t cache_maps(const CacheView &c, bool q4, int keys, CacheMaps *maps);

// Copies `box` rows from (page, row) on into shared memory; a page past the last
// reads as zeros.  Called by a whole, converged warp; one elected lane issues it
// (issued by several lanes each becomes a loop of some 80 clocks a copy).
__device__ __forceinline__ void plane_copy(const PlaneMap &p, uint32_t dst, uint32_t bar, int x,
                                           int c1, int c2, int c3)
{
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%3, %4, %5, %6}], [%2];\n}"
        ::"r"(dst), "l"(&p.m), "r"(bar), "r"(x), "r"(c1), "r"(c2), "r"(c3) : "memory");
}
// Row, head and page in the order of the map's axes.
__device__ __forceinline__ void plane_coords(const PlaneMap &p, int row, int head, int page, int *c1,
                                             int *c2, int *c3)
{
    *c1 = p.row_axis == 1 ? row : (p.head_axis == 1 ? head : page);
    *c2 = p.row_axis == 2 ? row : (p.head_axis == 2 ? head : page);
    *c3 = p.row_axis == 3 ? row : (p.head_axis == 3 ? head : page);
}

}  // namespace qkr
