// Device helpers of the paged cache.
#pragma once

#include "ff_launch.cuh"
#include "ff_paged.h"
#include "ff_ptx.cuh"

namespace ff {

// Pages of that many rows.
__device__ __forceinline__ int pages_of(const PagedState& s, int rows) { return (rows + (1 << s.shift) - 1) >> s.shift; }

// Page `i` of request r, whatever the table says.
__device__ __forceinline__ int page_at(const PagedState& s, int r, int i) {
  return clampi(__ldcg(s.tables + static_cast<size_t>(r) * s.width + i), 0, s.pages - 1);
}

// The last r < n with prefix[r] <= x, for prefix sums of n non-negative numbers, prefix[0] <= x < prefix[n]: the one that
// x falls into.
__device__ __forceinline__ int last_at_most(const int* prefix, int n, int x) {
  int lo = 0, hi = n;  // prefix[lo] <= x < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// A page's rows (or a few of them) of one head from a pool in groups of eight rows, [groups][D / 64][8][64]: `group` on.
__device__ __forceinline__ void tma_load_4d(void* smem_dst, const CUtensorMap* map, int group, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3}], [%4];"
      ::"r"(smem_u32(smem_dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(group), "r"(smem_u32(bar))
      : "memory");
}

}  // namespace ff
