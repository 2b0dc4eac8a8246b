// qb_order.cu -- the dispatch of a MoE layer: per-expert counts, offsets and
// the order of rows by expert, a stable counting sort of the top-k sets.
//
// The N*k entries are cut into runs, one CTA each.  The first launch stores
// every run's counts; in the second each CTA adds up all of them (16 bytes a
// load, all threads) to know where its run's entries of every expert start,
// and ranks the entries in order, 32 at a time: lanes with the same expert
// find each other (by ballots) and take consecutive places.  Its warps hold
// consecutive parts of the run, each with its own counters, in shared memory;
// the entries are read once, into registers, before the second launch waits
// for the first (a programmatic dependent of it).  No atomic decides a place,
// so equal inputs always give equal orders.  Latency bounds it, not the 12
// bytes of an entry: 131072 tokens x 6 of 256 experts 12.4 us, 7 tokens 4.2 us.
// (Putting a run in order in shared memory first, to write whole sectors, took
// 19 us: the two launches then no longer overlap.)
#include "qb_device.cuh"
#include "qb_internal.h"

namespace qb {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kRunMin = 4096;  // entries of a run at least: so few are one launch of one CTA
constexpr int kHold = 16;      // steps of 32 entries that a warp holds in registers

__global__ void __launch_bounds__(kThreads)
    order_count_kernel(const int32_t* __restrict__ topk, int64_t L, int E, int64_t run,
                       int* __restrict__ runs) {
  __shared__ int cnt[kMaxE];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int e = threadIdx.x; e < E; e += kThreads) cnt[e] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * run, hi = lo + run < L ? lo + run : L;
  for (int64_t i0 = lo + threadIdx.x; i0 < hi; i0 += kHold * kThreads) {
    int e[kHold];
#pragma unroll
    for (int j = 0; j < kHold; ++j)
      e[j] = i0 + j * kThreads < hi ? __ldg(topk + i0 + j * kThreads) : -1;
#pragma unroll
    for (int j = 0; j < kHold; ++j)
      if ((unsigned)e[j] < (unsigned)E) atomicAdd(cnt + e[j], 1);
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

// The lanes that hold the same expert (any of the lanes with -1 where this one
// does), by a ballot for each bit of it: match_any takes some 60 cycles of the
// whole SM, ten ballots a sixth of that.
__device__ __forceinline__ unsigned lanes_alike(int e, int bits) {
  unsigned same = __ballot_sync(0xffffffffu, e >= 0);
#pragma unroll
  for (int b = 0; b < 10; ++b) {
    if (b >= bits) break;
    const bool set = e >> b & 1;
    const unsigned with = __ballot_sync(0xffffffffu, set);
    same &= set ? with : ~with;
  }
  return same;
}

__global__ void __launch_bounds__(kThreads)
    order_place_kernel(const int32_t* __restrict__ topk, int64_t L, int E, int k, int64_t run,
                       int n_runs, const int* runs, int32_t* __restrict__ counts,
                       int32_t* __restrict__ offsets, int32_t* __restrict__ slot_of,
                       int32_t* __restrict__ token_of) {
  extern __shared__ int sm[];
  int* part = sm;                  // [kWarps][E]
  int* start = part + kWarps * E;  // [E] entries of each expert, then their first place
  int* before = start + E;         // [E] entries of earlier runs
  __shared__ int warp_sum[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t lo = blockIdx.x * run, hi = lo + run < L ? lo + run : L;
  const int64_t length = (run / kWarps + 31) / 32 * 32;  // of a warp's part
  int64_t wlo = lo + warp * length;
  if (wlo > hi) wlo = hi;
  const int64_t whi = warp == kWarps - 1 || wlo + length > hi ? hi : wlo + length;

  const auto read = [&](int64_t i0, int(&e)[kHold]) {
#pragma unroll
    for (int j = 0; j < kHold; ++j) {
      const int64_t i = i0 + 32 * j + lane;
      e[j] = i < whi ? __ldg(topk + i) : -1;
    }
#pragma unroll
    for (int j = 0; j < kHold; ++j)
      if ((unsigned)e[j] >= (unsigned)E) e[j] = -1;
  };
  int e[kHold];
  read(wlo, e);
  for (int i = threadIdx.x; i < (kWarps + 2) * E; i += kThreads) sm[i] = 0;
  __syncthreads();
  int* next = part + warp * E;
  const int bits = 32 - __clz(E - 1);
  for (int64_t i0 = wlo; i0 < whi; i0 += 32 * kHold) {
    if (i0 != wlo) read(i0, e);
#pragma unroll
    for (int j = 0; j < kHold; ++j)
      if (e[j] >= 0) atomicAdd(next + e[j], 1);
  }
  if (n_runs > 1) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // four experts of a thread, the runs dealt out over the threads
    const int quads = E / 4, q = threadIdx.x % quads, parts = kThreads / quads;
    int4 all = make_int4(0, 0, 0, 0), mine = all;
    if (threadIdx.x < parts * quads) {
      for (int c0 = threadIdx.x / quads; c0 < n_runs; c0 += 8 * parts) {
        int4 n[8];  // eight reads in flight, to the last
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = c0 + j * parts;
          n[j] = make_int4(0, 0, 0, 0);
          if (c < n_runs) n[j] = __ldcg(reinterpret_cast<const int4*>(runs + (int64_t)c * E) + q);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          all.x += n[j].x;
          all.y += n[j].y;
          all.z += n[j].z;
          all.w += n[j].w;
          if (c0 + j * parts < (int)blockIdx.x) {
            mine.x += n[j].x;
            mine.y += n[j].y;
            mine.z += n[j].z;
            mine.w += n[j].w;
          }
        }
      }
      atomicAdd(start + 4 * q, all.x);
      atomicAdd(start + 4 * q + 1, all.y);
      atomicAdd(start + 4 * q + 2, all.z);
      atomicAdd(start + 4 * q + 3, all.w);
      atomicAdd(before + 4 * q, mine.x);
      atomicAdd(before + 4 * q + 1, mine.y);
      atomicAdd(before + 4 * q + 2, mine.z);
      atomicAdd(before + 4 * q + 3, mine.w);
    }
  } else {
    __syncthreads();
    for (int x = threadIdx.x; x < E; x += kThreads)
      for (int w = 0; w < kWarps; ++w) start[x] += part[w * E + x];
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int x = threadIdx.x; x < E; x += kThreads) counts[x] = start[x];
  __syncthreads();
  const int total = exclusive_sums(start, E, warp_sum);
  for (int x = threadIdx.x; x < E; x += kThreads) {
    if (blockIdx.x == 0) offsets[x] = start[x];
    int at = start[x] + before[x];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {  // counts -> first place of each warp's entries
      const int n = part[w * E + x];
      part[w * E + x] = at;
      at += n;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) offsets[E] = total;
  __syncthreads();
  for (int64_t i0 = wlo; i0 < whi; i0 += 32 * kHold) {
    if (whi - wlo > 32 * kHold) read(i0, e);
#pragma unroll
    for (int j = 0; j < kHold; ++j) {
      const int64_t i = i0 + 32 * j + lane;
      if (i - lane >= whi) break;
      const unsigned same = lanes_alike(e[j], bits);
      const int rank = __popc(same & ((1u << lane) - 1u));
      int slot = -1;
      if (e[j] >= 0) slot = next[e[j]] + rank;
      __syncwarp();
      if (e[j] >= 0 && rank == 0) next[e[j]] += __popc(same);
      __syncwarp();
      if (i < whi) {
        slot_of[i] = slot;
        if (slot >= 0) token_of[slot] = (int32_t)((uint32_t)i / (uint32_t)k);
      }
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
  if (n_runs <= 1) {
    order_place_kernel<<<1, kThreads, smem, stream>>>(topk, L, E, k, run, 1, runs, counts, offsets,
                                                      slot_of, token_of);
    return launch_status();
  }
  order_count_kernel<<<n_runs, kThreads, 0, stream>>>(topk, L, E, run, runs);
  const int st = launch_status();
  if (st != QB_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)n_runs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, order_place_kernel, topk, L, E, k, run, n_runs,
                         static_cast<const int*>(runs), counts, offsets, slot_of,
                         token_of) != cudaSuccess) {
    (void)cudaGetLastError();
    return QB_ECUDA;
  }
  return launch_status();
}

}  // namespace qb
