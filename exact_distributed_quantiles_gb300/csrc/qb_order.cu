// qb_order.cu -- the dispatch of a MoE layer: per-expert counts, offsets and
// the order of rows by expert, a stable counting sort of the top-k sets.
//
// The N*k entries are cut into runs, one CTA each.  A CTA counts its entries
// by expert (its warps hold consecutive parts of the run, each with its own
// counters); the first launch stores the runs' counts, the second reads all
// of them to know where its run's entries of every expert start, and ranks
// the entries in order, 32 at a time: lanes with the same expert find each
// other (match_any) and take consecutive places.  No atomic decides a place,
// so equal inputs always give equal orders.
#include "qb_device.cuh"
#include "qb_internal.h"

namespace qb {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kRunMin = 4096;  // entries of a run at least: one CTA alone below twice that

// Counts of the warp's part of the run into its own counters.
__device__ __forceinline__ void count_part(const int32_t* topk, int64_t lo, int64_t hi, int E,
                                           int* mine) {
  for (int64_t i = lo + (threadIdx.x & 31); i < hi; i += 32) {
    const int e = topk[i];
    if ((unsigned)e < (unsigned)E) atomicAdd(mine + e, 1);
  }
}

struct Run {
  int64_t lo, hi;      // the CTA's entries
  int64_t wlo, whi;    // this warp's
};
__device__ __forceinline__ Run run_of(int64_t L, int64_t run) {
  Run r;
  r.lo = blockIdx.x * run;
  r.hi = r.lo + run < L ? r.lo + run : L;
  const int64_t part = (run / kWarps + 31) / 32 * 32;
  const int warp = threadIdx.x >> 5;
  r.wlo = r.lo + warp * part;
  if (r.wlo > r.hi) r.wlo = r.hi;
  r.whi = warp == kWarps - 1 || r.wlo + part > r.hi ? r.hi : r.wlo + part;
  return r;
}

__global__ void __launch_bounds__(kThreads)
    order_count_kernel(const int32_t* __restrict__ topk, int64_t L, int E, int64_t run,
                       int* __restrict__ runs) {
  __shared__ int cnt[kMaxE];
  for (int e = threadIdx.x; e < E; e += kThreads) cnt[e] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * run, hi = lo + run < L ? lo + run : L;
  for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) {
    const int e = topk[i];
    if ((unsigned)e < (unsigned)E) atomicAdd(cnt + e, 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kThreads) runs[(int64_t)blockIdx.x * E + e] = cnt[e];
}

// E <= 1024 counts -> their exclusive sums, in place in shared memory; every
// thread of the CTA calls it.  Returns the total.
__device__ __forceinline__ int exclusive_sums(int* v, int E, int* warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kPer = kMaxE / kThreads;
  int x[kPer], s = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = kPer * threadIdx.x + i;
    x[i] = e < E ? v[e] : 0;
    s += x[i];
  }
  int inc = s;
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += u;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int before = 0, total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  int at = before + inc - s;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = kPer * threadIdx.x + i;
    if (e < E) v[e] = at;
    at += x[i];
  }
  __syncthreads();
  return total;
}

__global__ void __launch_bounds__(kThreads)
    order_place_kernel(const int32_t* __restrict__ topk, int64_t L, int E, int k, int64_t run,
                       int n_runs, const int* __restrict__ runs, int32_t* __restrict__ counts,
                       int32_t* __restrict__ offsets, int32_t* __restrict__ slot_of,
                       int32_t* __restrict__ token_of) {
  extern __shared__ int sm[];
  int* part = sm;                  // [kWarps][E]
  int* start = part + kWarps * E;  // [E] first place of each expert, then of this run's entries
  int* before = start + E;         // [E] entries of earlier runs
  __shared__ int warp_sum[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Run r = run_of(L, run);
  for (int i = threadIdx.x; i < kWarps * E; i += kThreads) part[i] = 0;
  __syncthreads();
  count_part(topk, r.wlo, r.whi, E, part + warp * E);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kThreads) {
    int all = 0, mine = 0;
    if (n_runs > 1) {
#pragma unroll 8
      for (int c = 0; c < n_runs; ++c) {
        const int n = runs[(int64_t)c * E + e];
        all += n;
        mine += c < (int)blockIdx.x ? n : 0;
      }
    } else {
      for (int w = 0; w < kWarps; ++w) all += part[w * E + e];
    }
    start[e] = all;
    before[e] = mine;
    if (blockIdx.x == 0) counts[e] = all;
  }
  __syncthreads();
  const int total = exclusive_sums(start, E, warp_sum);
  for (int e = threadIdx.x; e < E; e += kThreads) {
    if (blockIdx.x == 0) offsets[e] = start[e];
    int at = start[e] + before[e];
    for (int w = 0; w < kWarps; ++w) {  // counts -> first place of each warp's entries
      const int n = part[w * E + e];
      part[w * E + e] = at;
      at += n;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) offsets[E] = total;
  __syncthreads();
  int* next = part + warp * E;
  for (int64_t i0 = r.wlo; i0 < r.whi; i0 += 32) {
    const int64_t i = i0 + lane;
    int e = -1;
    if (i < r.whi) e = topk[i];
    if ((unsigned)e >= (unsigned)E) e = -1;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int slot = -1;
    if (e >= 0) slot = next[e] + rank;
    __syncwarp();
    if (e >= 0 && rank == 0) next[e] += __popc(same);
    __syncwarp();
    if (i < r.whi) {
      slot_of[i] = slot;
      if (slot >= 0) token_of[slot] = (int32_t)(i / k);
    }
  }
  // places that no entry takes (dropped entries): -1
  for (int64_t i = total + (int64_t)blockIdx.x * kThreads + threadIdx.x; i < L;
       i += (int64_t)gridDim.x * kThreads)
    token_of[i] = -1;
}

int64_t run_length(int64_t L) {
  const int64_t sms = sm_count();
  int64_t run = (L + sms - 1) / sms;
  run = (run + 511) / 512 * 512;
  return run < kRunMin ? kRunMin : run;
}

}  // namespace

int64_t order_workspace_bytes(int64_t N, int E, int k) {
  const int64_t run = run_length(N * k);
  return (N * k + run - 1) / run * E * 4;
}

int launch_expert_order(const int32_t* topk, int64_t N, int E, int k, int32_t* counts,
                        int32_t* offsets, int32_t* slot_of, int32_t* token_of, void* workspace,
                        cudaStream_t stream) {
  const int64_t L = N * k, run = run_length(L);
  const int n_runs = (int)((L + run - 1) / run);
  int* runs = static_cast<int*>(workspace);
  const int smem = (kWarps + 2) * E * 4;
  static std::atomic<uint64_t> done{0};
  if (!smem_attribute(order_place_kernel, (kWarps + 2) * kMaxE * 4, done)) return launch_status();
  if (n_runs > 1) {
    order_count_kernel<<<n_runs, kThreads, 0, stream>>>(topk, L, E, run, runs);
    const int st = launch_status();
    if (st != QB_OK) return st;
  }
  order_place_kernel<<<n_runs < 1 ? 1 : n_runs, kThreads, smem, stream>>>(
      topk, L, E, k, run, n_runs, runs, counts, offsets, slot_of, token_of);
  return launch_status();
}

}  // namespace qb
