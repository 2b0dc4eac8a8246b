// qb_groups.cuh -- rows in groups (experts), as offsets on the device describe
// them: shared by the token-major quantiser and the experts' products, which
// have to number a group's units alike.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace qb {

// Rows first .. end - 1 of group g, held within [0, rows] whatever offsets
// says; nullptr: one group of all rows.
__device__ __forceinline__ void group_rows(const int32_t* offsets, int g, int64_t rows,
                                           int64_t& first, int64_t& end) {
  first = 0;
  end = rows;
  if (offsets) {
    first = __ldg(offsets + g);
    end = __ldg(offsets + g + 1);
    first = first < 0 ? 0 : first > rows ? rows : first;
    end = end < first ? first : end > rows ? rows : end;
  }
}

// pre[g] = units of `unit` rows (the last of a group may be short) of the
// groups before g, g = 0 .. G, in shared memory.  Every thread of the CTA calls
// it, and a barrier has to follow.
__device__ __forceinline__ void count_units(const int32_t* offsets, int G, int64_t rows, int unit,
                                            int* pre) {
  const int lane = threadIdx.x & 31;
  for (int g = threadIdx.x; g < G; g += (int)blockDim.x) {
    int64_t first, end;
    group_rows(offsets, g, rows, first, end);
    pre[g + 1] = (int)((end - first + unit - 1) / unit);
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

}  // namespace qb
