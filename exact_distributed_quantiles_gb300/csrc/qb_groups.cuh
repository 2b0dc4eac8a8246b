// qb_groups.cuh -- rows in groups (experts), as offsets on the device describe
// them: shared by the token-major quantiser and the experts' products, which
// have to number a group's units alike.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace qb {

// start[g] = first row of group g, g = 0 .. G, held within [0, rows] whatever
// offsets says (nullptr: one group of all rows); pre[g] = units of `unit` rows
// (the last of a group may be short) of the groups before g.  Both in shared
// memory.  Every thread of the CTA calls it, and a barrier has to follow.
__device__ __forceinline__ void count_units(const int32_t* offsets, int G, int rows, int unit,
                                            int* start, int* pre) {
  const int lane = threadIdx.x & 31;
  const auto first_row = [&](int g) {
    int v = g == 0 ? 0 : rows;
    if (offsets) v = __ldg(offsets + g);
    return v < 0 ? 0 : v > rows ? rows : v;
  };
  for (int g = threadIdx.x; g < G; g += (int)blockDim.x) {
    const int first = first_row(g), end = first_row(g + 1);
    start[g] = first;
    if (g == G - 1) start[G] = end;
    pre[g + 1] = end > first ? (end - first + unit - 1) / unit : 0;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int carry = 0;
    for (int g0 = 0; g0 < G; g0 += 32) {
      int v = g0 + lane < G ? pre[g0 + lane + 1] : 0;
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += u;
      }
      // offsets that do not ascend could add up without end: the sum stops at 2^30
      v = carry + v < (1 << 30) ? carry + v : 1 << 30;
      if (g0 + lane < G) pre[g0 + lane + 1] = v;
      carry = __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) pre[0] = 0;
  }
}

// The group of unit u: the last one whose first unit is not behind it.
__device__ __forceinline__ int group_of(const int* pre, int G, int u) {
  int lo = 0, hi = G - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= u) lo = mid; else hi = mid - 1;
  }
  return lo;
}

}  // namespace qb
