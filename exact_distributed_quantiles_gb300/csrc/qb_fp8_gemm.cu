// qb_fp8_gemm.cu -- the experts' products on 8-bit floating-point operands
// with one power-of-two scale for each 128 values of the contraction
// (qb_fp8.cu makes them), on the 5th-generation tensor cores.
//
//   rows   out[r, n]    = sum_k A[r, k] B[g, n, k],     offsets[g] <= r < offsets[g+1]
//   cols   out[g, n, k] = sum_t A[n, t] B[k, t],        t over group g's columns
//
// A and B are e4m3 codes with scales 2^(byte - 127); the block-scaled MMA
// (kind::mxf8f6f4, one e8m0 scale per 32 values of K) multiplies by the scales
// itself, so a product costs no more than unscaled 8-bit codes and the
// accumulator, fp32 in tensor memory, is read once.  The scale of a 128-value
// block serves the four MMAs of that block.
//
// B is the MMA's M side and A its N side, D = B A^T: the output's contiguous
// index runs along the lanes of tensor memory, so a warp's store of one column
// of D is one contiguous piece of an output row; and the N side takes any
// multiple of 16, so a group's rows are cut into equal tiles that fit it
// (ragged groups cost at most 15 rows each, not 127).
//
// A pair of CTAs (cluster of 2, cta_group::2) computes 256 x n outputs, n up
// to 224: each CTA loads its 128 rows of B and half of A's rows, 30 KB for
// 128 values of K instead of the 44 KB that one CTA's 128 x 224 tile takes.
// One persistent pair per two SMs:
//   warp 0      TMA producer of its CTA (128-byte swizzle, seven stages); both
//               CTAs' copies count on the first CTA's barrier;
//   warp 1      TMEM; in the first CTA one lane copies four K blocks' scales
//               to both CTAs' tensor memory at a time (tcgen05.cp) and issues
//               four MMAs per K block for the pair;
//   warps 2-3   the scales' producers: one 32-bit word holds a row's scales of
//               four K blocks, laid out as tcgen05.cp wants them;
//   warps 4-11  the epilogue of one accumulator while the other is filled.
// The rows of a group are known on the device only: each CTA sums the groups'
// tile counts itself, so the host never waits for the dispatch.
// Measured: 98304 rows x 2048 -> 1024 over 256 experts 173 us (2.4 PFLOP/s, 5.4
// TB/s; 197 us back to back, at the power limit's 1.3 GHz), 48 rows 23 us (HBM
// and 2.3 rounds of tiles), weight gradient of 64 experts 1024 x 2048 from
// 65536 tokens 152 us (the SM's way out: output stores and operand requests).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "qb_device.cuh"
#include "qb_groups.cuh"
#include "qb_internal.h"
#include "qb_tc.cuh"

namespace qb {
namespace {

constexpr int kBP = 256;   // rows of B (outputs along a row) of a pair's tile
constexpr int kBQ = 224;   // rows of A at most
constexpr int kBK = 128;   // bytes of K per stage: one swizzle row
constexpr int kStages = 7;
constexpr int kPBytes = kBP / 2 * kBK;
constexpr int kStageBytes = kPBytes + kBQ / 2 * kBK;
constexpr int kSfStages = 4;
constexpr int kSfBytes = 512 + 1024;  // scales of 128 rows of B and of 256 rows of A
constexpr int kThreads = 12 * 32;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kScaleCol = 2 * kBQ;  // accumulators below, scales from here
constexpr int kSmem = 1024 + kStages * kStageBytes + kSfStages * kSfBytes + 512 /*barriers*/ +
                      2 * 4 * (kMaxGroups + 4);
constexpr int kStartAt = kMaxGroups + 4;  // the groups' first rows, behind their units' sums

struct Args {
  const uint8_t* sp;
  const uint8_t* sq;
  const int32_t* offsets;  // nullptr: one group
  void* out;
  int64_t tokens;  // what offsets is clamped to
  int P;           // rows of B: outputs along a row
  int Q;           // cols mode: rows of A
  int kblocks;     // K blocks of every tile (rows mode), of the operands (cols mode)
  int G;
  int bq;          // most rows of A in a tile, a multiple of 16
  int np;          // tiles along B's rows
  int nq, part;    // cols mode: tiles along A's rows, rows of each
  int pitch_p, pitch_q;
  int p_blocks;    // rows mode: scale rows of B per group
  int f32, accumulate;
  int* status;
};

// ---- the pair's instructions (cta_group::2)
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// One lane of the (converged) warp, always the same: the compiler knows then
// that a single thread issues, and keeps the operands of the instructions
// below, which are the same in all lanes, in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// The address of the first CTA's copy of a shared-memory variable.
__device__ __forceinline__ uint32_t in_first(uint32_t saddr) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(saddr));
  return a;
}
__device__ __forceinline__ void tmem_alloc2(uint32_t dst_smem) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
               "r"(kTmemCols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(kTmemCols)
               : "memory");
}
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc,
                                           uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X"
      " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// 32 rows x 16 bytes of each CTA's shared memory -> 4 columns of its tensor
// memory, the same in each of the four groups of 32 lanes.
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint32_t smem) {
  uint64_t d = 0;
  d |= (uint64_t)((smem & 0x3FFFFu) >> 4);
  d |= (uint64_t)(128 >> 4) << 32;  // 8 rows of 16 bytes to the next 8
  d |= (uint64_t)1 << 46;
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(d) : "memory");
}
// Arrives on the barrier at this offset in both CTAs once the MMAs and copies
// issued so far are done.
__device__ __forceinline__ void commit_both(uint32_t mbar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(mbar),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                        uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
      ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(mbar)
      : "memory");
}
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                        uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile"
      ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(mbar)
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// Orders between the CTAs of a pair name the cluster's scope.  All data that
// passes so (tiles, scales) lies in shared memory, so the fences order accesses
// to shared memory alone: a plain release to the cluster would wait for the
// thread's global loads and stores too, and a plain acquire costs more at every
// stage.  Against orders of the CTA's scope, which do not reach the other CTA:
// weight gradient of 64 experts, 65536 tokens, 165 -> 166 us (plain ones 169 ->
// 177), product of 98304 rows 201 -> 196 us (206 -> 210), of 48 rows 24.4 ->
// 23.0 us (24.5 -> 26.7).
__device__ __forceinline__ void fence_release_smem() {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
}
__device__ __forceinline__ void fence_acquire_smem() {
  asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
}
// Arrives on the first CTA's barrier: after fence_release_smem where it
// publishes shared memory (the scales), by itself where it only says that
// tensor memory has been read (the epilogue, after tcgen05.fence).
__device__ __forceinline__ void arrive_first(uint32_t mbar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(mbar)
               : "memory");
}
// mbar_wait_bounded by a whole warp, with the same result in all lanes: for
// what the tensor core alone did to tensor memory (a tcgen05 fence follows).
__device__ __forceinline__ bool try_wait_warp(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return __all_sync(0xffffffffu, ok != 0);
}
__device__ __forceinline__ bool wait_tmem(uint32_t bar, uint32_t parity, int* status) {
  if (try_wait_warp(bar, parity)) return true;
  for (uint32_t it = 0; it < 1u << 24; ++it) {
    if (try_wait_warp(bar, parity)) return true;
    if (it > 64) __nanosleep(64);
  }
  if ((threadIdx.x & 31) == 0) atomicOr(status, kDevTimeout);
  return false;
}
// The same for buffers in shared memory, filled or used up.
__device__ __forceinline__ bool wait_smem(uint32_t bar, uint32_t parity, int* status) {
  const bool ok = wait_tmem(bar, parity, status);
  fence_acquire_smem();
  return ok;
}

// A place in a ring of n buffers, and the parity of its round.
template <int n>
struct Ring {
  uint32_t at = 0, parity = 0;
  __device__ __forceinline__ void next() {
    if (++at == n) {
      at = 0;
      parity ^= 1u;
    }
  }
};

// Instruction descriptor, kind::mxf8f6f4: both operands e4m3 (format 0) and
// K-major, N >> 3 at bits 17-22, scales e8m0 (bit 23), M >> 4 at bits 24-28;
// the byte of a scale word that serves this MMA at bits 29-30 (M side) and
// 4-5 (N side).
__device__ __forceinline__ uint32_t idesc_of(int n, uint32_t byte) {
  return ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(kBP >> 4) << 24) | (byte << 29) |
         (byte << 4);
}

// One tile of the walk.
struct Tile {
  int g;         // group
  int q0;        // first row of A
  int rows;      // rows of A that are stored
  int n;         // the MMA's N: rows rounded up to 16
  int p0;        // first row of B
  int kb0, kb1;  // K blocks
};

// Every role walks the tiles by itself, so this stays short: 32-bit numbers
// (the host bounds the tiles), three divisions and a search in shared memory.
template <bool kCols>
__device__ __forceinline__ Tile tile_at(const Args& a, const int* pre, uint32_t t) {
  const int* start = pre + kStartAt;
  Tile r;
  const uint32_t m = t / (uint32_t)a.np;
  r.p0 = (int)(t - m * (uint32_t)a.np) * kBP;
  uint32_t first, end, i;
  if (kCols) {
    r.g = (int)(m / (uint32_t)a.nq);
    i = m - (uint32_t)r.g * (uint32_t)a.nq;
    first = 0;
    end = (uint32_t)a.Q;
    r.kb0 = pre[r.g] < a.kblocks ? pre[r.g] : a.kblocks;
    r.kb1 = pre[r.g + 1] < a.kblocks ? pre[r.g + 1] : a.kblocks;
  } else {
    r.g = group_of(pre, a.G, (int)m);
    i = m - (uint32_t)pre[r.g];
    first = (uint32_t)start[r.g];
    end = (uint32_t)(start[r.g + 1] > start[r.g] ? start[r.g + 1] : start[r.g]);
    r.kb0 = 0;
    r.kb1 = a.kblocks;
  }
  // the group's rows in equal parts, each a multiple of 16 but for the last
  const uint32_t count = end - first;
  uint32_t part = (uint32_t)a.part;
  if (!kCols) {
    const uint32_t parts = count > 0 ? (count + (uint32_t)a.bq - 1) / (uint32_t)a.bq : 1u;
    part = ((count + parts - 1) / parts + 15u) & ~15u;
  }
  r.q0 = (int)(first + i * part);
  const int left = (int)end - r.q0 < (int)part ? (int)end - r.q0 : (int)part;
  r.rows = left > 0 ? left : 0;
  r.n = r.rows > 0 ? (r.rows + 15) & ~15 : 16;
  return r;
}

// Sums of at most this many K blocks are left to the accumulator: the tensor
// core truncates as it adds, and its error grows with the number of its steps
// (measured against 64 bits: 4e-7 of the result's norm at 2048 values of K,
// 6e-6 at 15000); longer sums are continued in registers, rounded to nearest.
constexpr int kSegment = 16;
__device__ __forceinline__ int segments_of(const Tile& w) {
  const int n = (w.kb1 - w.kb0 + kSegment - 1) / kSegment;
  return n > 0 ? n : 1;
}

// Stores 32 columns of D: a lane holds one output of each of 32 rows, so a
// warp's store is one contiguous piece of a row.
template <bool kCols>
__device__ __forceinline__ void store_rows(const Args& a, const uint32_t (&v)[32], int64_t at,
                                           int rows) {
  if (a.f32) {
    float* out = reinterpret_cast<float*>(a.out) + at;
    if (kCols && a.accumulate) {  // products only write
#pragma unroll
      for (int j = 0; j < 32; j += 4) {  // four reads in flight
        float old[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j + i < rows) old[i] = out[(int64_t)(j + i) * a.P];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j + i < rows) out[(int64_t)(j + i) * a.P] = old[i] + __uint_as_float(v[j + i]);
      }
    } else if (rows >= 32) {
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        *out = __uint_as_float(v[j]);
        out += a.P;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < rows) out[(int64_t)j * a.P] = __uint_as_float(v[j]);
    }
  } else {
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + at;
    if (rows >= 32) {
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        *out = __float2bfloat16_rn(__uint_as_float(v[j]));
        out += a.P;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < rows) out[(int64_t)j * a.P] = __float2bfloat16_rn(__uint_as_float(v[j]));
    }
  }
}

// A warp's walk over its pair's tiles.  Finding a tile takes a search and
// divisions, a thousand cycles and more of latency; the lanes find 32 tiles at
// once, and each tile is then handed round by shuffles (whose results the
// compiler knows to be the same in all lanes).
template <bool kCols>
struct Walk {
  const Args& a;
  const int* pre;
  uint32_t t, step, n_tiles;
  int i = 32;
  Tile mine;
  __device__ __forceinline__ Walk(const Args& a_, const int* pre_, uint32_t t0, uint32_t step_,
                                  uint32_t n)
      : a(a_), pre(pre_), t(t0), step(step_), n_tiles(n) {}
  // The next tile; false behind the last one.
  __device__ __forceinline__ bool next(Tile& w) {
    if (t >= n_tiles) return false;
    if (i == 32) {
      const uint64_t u = (uint64_t)t + (uint64_t)step * (threadIdx.x & 31);
      if (u < n_tiles) mine = tile_at<kCols>(a, pre, (uint32_t)u);
      i = 0;
      __syncwarp();
    }
    w.g = __shfl_sync(0xffffffffu, mine.g, i);
    w.q0 = __shfl_sync(0xffffffffu, mine.q0, i);
    w.rows = __shfl_sync(0xffffffffu, mine.rows, i);
    w.n = __shfl_sync(0xffffffffu, mine.n, i);
    w.p0 = __shfl_sync(0xffffffffu, mine.p0, i);
    w.kb0 = __shfl_sync(0xffffffffu, mine.kb0, i);
    w.kb1 = __shfl_sync(0xffffffffu, mine.kb1, i);
    ++i;
    t = step < n_tiles - t ? t + step : n_tiles;
    return true;
  }
};

template <bool kCols>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap map_p,
                    const __grid_constant__ CUtensorMap map_q32,
                    const __grid_constant__ CUtensorMap map_q8, const Args a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* sbase = smem_raw + (base - raw);
  unsigned char* sf = sbase + kStages * kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sf + kSfStages * kSfBytes);
  uint64_t* empty = full + kStages;
  uint64_t* sf_full = empty + kStages;
  uint64_t* sf_empty = sf_full + kSfStages;
  uint64_t* tfull = sf_empty + kSfStages;
  uint64_t* tempty = tfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  int* pre = reinterpret_cast<int*>(reinterpret_cast<unsigned char*>(full) + 512);

  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();

  if (threadIdx.x == 32 * 4) {
    prefetch_map(&map_p);
    prefetch_map(&map_q32);
    prefetch_map(&map_q8);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int s = 0; s < kSfStages; ++s) {
      mbar_init(sf_full + s, 2);  // one producer of each CTA
      mbar_init(sf_empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull + b, 1);
      mbar_init(tempty + b, 2 * 8);  // the epilogue's warps of both CTAs
    }
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc2(smem_u32(tmem_slot));
  tc_fence_before();
  cluster_arrive_release();  // this CTA's barriers and tensor memory are ready
  // tiles (rows mode) or 128-column blocks (cols mode) of the groups
  count_units(a.offsets, a.G, (int)a.tokens, kCols ? 128 : a.bq, pre + kStartAt, pre);
  __syncwarp();
  cluster_wait();  // the other CTA's are
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // more tiles than 2^31 - 1 only come of offsets that do not ascend
  const int64_t all = (int64_t)a.np * (kCols ? (int64_t)a.G * a.nq : (int64_t)pre[a.G]);
  const uint32_t n_tiles = all < INT32_MAX ? (uint32_t)all : (uint32_t)INT32_MAX;
  Walk<kCols> walk(a, pre, blockIdx.x >> 1, gridDim.x >> 1, n_tiles);

  // Every role's loop below is short on purpose: a warp alone issues an
  // instruction every few cycles, and 128 values of K last 400.
  if (warp == 0) {
    Ring<kStages> ring;
    uint32_t used = 0;  // stages filled so far, up to kStages
    bool ok = true;
    const uint32_t bar0 = smem_u32(empty);
    const uint32_t first_full = (uint32_t)uniform((int)in_first(smem_u32(full)));
    Tile w;
    while (ok && walk.next(w)) {
      // each CTA's rows of A, a multiple of 8: in boxes of 32, the last of
      // them back from the end (it repeats rows of the one before), or of 8
      const int half = w.n >> 1, q0 = w.q0 + (int)rank * half;
      const int p0 = w.p0 + (int)rank * (kBP / 2), z = kCols ? 0 : w.g;
      const int boxes = half >= 32 ? (half + 31) >> 5 : half >> 3;
      const uint32_t bytes = (uint32_t)(2 * kPBytes + 2 * boxes * (half >= 32 ? 32 : 8) * kBK);
      for (int kb = w.kb0; kb < w.kb1; ++kb) {
        if (used == (uint32_t)kStages) {
          ok = wait_smem(bar0 + 8u * ring.at, ring.parity ^ 1u, a.status);
          if (!ok) break;
        } else {
          ++used;
        }
        if (elect_one()) {
          const uint32_t dst = base + ring.at * (uint32_t)kStageBytes;
          const uint32_t bar = first_full + 8u * ring.at;
          const int x = kb * kBK;
          if (rank == 0) mbar_arrive_expect_tx(full + ring.at, bytes);
          load_3d(dst, &map_p, x, p0, z, bar);
          if (half >= 32) {
            for (int r = 0; r < half; r += 32) {
              const int at = r + 32 <= half ? r : half - 32;
              load_2d(dst + kPBytes + at * kBK, &map_q32, x, q0 + at, bar);
            }
          } else {
            for (int r = 0; r < half; r += 8)
              load_2d(dst + kPBytes + r * kBK, &map_q8, x, q0 + r, bar);
          }
        }
        __syncwarp();
        ring.next();
      }
    }
    // Leave no copy of either CTA in flight, whatever the MMAs came to: the
    // last fill of every stage, oldest first.  After a full walk they have all
    // been used, and nothing is waited for.
    if (rank == 0) {
      if (used < (uint32_t)kStages) ring = Ring<kStages>{0, 1u};
      for (uint32_t i = 0; i < used; ++i) {
        wait_smem(smem_u32(full) + 8u * ring.at, ring.parity ^ 1u, a.status);
        ring.next();
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      Ring<kStages> ring;
      Ring<kSfStages> sring;
      Ring<2> acc;
      uint32_t fresh = 2;  // accumulators not used before
      const uint32_t taddr = (uint32_t)uniform((int)tmem);
      const uint32_t sfa = taddr + kScaleCol, sfb = sfa + 4;
      const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
      const uint32_t sf_full0 = smem_u32(sf_full), sf_empty0 = smem_u32(sf_empty);
      const uint32_t tfull0 = smem_u32(tfull), tempty0 = smem_u32(tempty);
      bool ok = true;
      Tile w;
      while (ok && walk.next(w)) {
        const int segments = segments_of(w);
        const uint32_t idesc0 = idesc_of(w.n, 0);
        int kb = w.kb0;
        for (int seg = 0; seg < segments && ok; ++seg) {
          if (fresh > 0)
            --fresh;
          else
            ok = wait_tmem(tempty0 + 8u * acc.at, acc.parity ^ 1u, a.status);
          if (!ok) break;
          const uint32_t d = taddr + acc.at * (uint32_t)kBQ;
          const int end = w.kb1 - kb < kSegment ? w.kb1 : kb + kSegment;
          uint32_t more = 0;
          while (kb < end && ok) {  // a step: up to four K blocks of one scale word
            const int stop = (kb | 3) + 1 < end ? (kb | 3) + 1 : end;
            if (kb == w.kb0 || (kb & 3) == 0) {
              ok = wait_smem(sf_full0 + 8u * sring.at, sring.parity, a.status);
              if (!ok) break;
              tc_fence_after();
              if (elect_one()) {
                const uint32_t src = smem_u32(sf) + sring.at * (uint32_t)kSfBytes;
                copy_scales(sfa, src);
                copy_scales(sfb, src + 512);
                if (w.n > 128) copy_scales(sfb + 4, src + 1024);
                commit_both(sf_empty0 + 8u * sring.at);
              }
              __syncwarp();
              sring.next();
            }
            for (; kb < stop; ++kb) {
              ok = wait_smem(full0 + 8u * ring.at, ring.parity, a.status);
              if (!ok) break;
              tc_fence_after();
              if (elect_one()) {
                const uint64_t dp = smem_desc_sw128(base + ring.at * (uint32_t)kStageBytes);
                const uint64_t dq = dp + (uint64_t)(kPBytes >> 4);
                const uint32_t idesc = idesc0 | (uint32_t)(kb & 3) << 29 | (uint32_t)(kb & 3) << 4;
                // 32 values of K at a time, 32 bytes (two address units) along the row
                mma_scaled(d, dp, dq, idesc, sfa, sfb, more);
                mma_scaled(d, dp + 2, dq + 2, idesc, sfa, sfb, 1u);
                mma_scaled(d, dp + 4, dq + 4, idesc, sfa, sfb, 1u);
                mma_scaled(d, dp + 6, dq + 6, idesc, sfa, sfb, 1u);
                commit_both(empty0 + 8u * ring.at);
              }
              __syncwarp();
              more = 1;
              ring.next();
            }
          }
          if (ok && elect_one()) commit_both(tfull0 + 8u * acc.at);
          __syncwarp();
          acc.next();
        }
      }
    }
  } else if (warp == 2 || warp == 3) {
    // Warp 2 serves the even steps of four K blocks, warp 3 the odd ones; each
    // reads its next step's words while the current one waits for its place.
    uint32_t vp[4], vq[8];
    Tile w;
    int c = 0, c_end = 0;  // steps of tile w: [c, c_end)
    uint32_t gs = 0;       // steps before (w, c)
    const auto settle = [&]() {  // the next step of this warp at or after (w, c)
      for (;;) {
        while (c >= c_end) {
          if (!walk.next(w)) return false;
          c = w.kb0 >> 2;
          c_end = w.kb0 < w.kb1 ? (w.kb1 + 3) >> 2 : c;
        }
        if ((gs & 1u) == (uint32_t)(warp - 2)) return true;
        ++c;
        ++gs;
      }
    };
    const auto read = [&]() {
      // lane l holds rows l, l + 32, l + 64 and l + 96 of each 128
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = w.p0 + (int)rank * (kBP / 2) + 32 * j + (kCols ? lane : 0);
        const int64_t row = kCols ? p : (int64_t)w.g * a.p_blocks + (p >> 7);
        vp[j] = p < a.P ? __ldg(reinterpret_cast<const uint32_t*>(a.sp + row * a.pitch_p + 4 * c))
                        : 0u;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = lane + 32 * j;
        vq[j] = r < w.rows ? __ldg(reinterpret_cast<const uint32_t*>(
                                 a.sq + (int64_t)(w.q0 + r) * a.pitch_q + 4 * c))
                           : 0u;
      }
    };
    bool more = settle();
    if (more) read();
    while (more) {
      const uint32_t at = gs;
      const uint4 wp = make_uint4(vp[0], vp[1], vp[2], vp[3]);
      const uint4 w0 = make_uint4(vq[0], vq[1], vq[2], vq[3]);
      const uint4 w1 = make_uint4(vq[4], vq[5], vq[6], vq[7]);
      ++c;
      ++gs;
      more = settle();
      if (more) read();
      const int s = (int)(at % kSfStages);
      if (at >= (uint32_t)kSfStages &&
          !wait_smem(smem_u32(sf_empty + s), (at / kSfStages - 1) & 1u, a.status))
        break;
      uint4* dst = reinterpret_cast<uint4*>(sf + s * kSfBytes) + lane;
      dst[0] = wp;
      dst[32] = w0;
      dst[64] = w1;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        fence_release_smem();
        arrive_first(in_first(smem_u32(sf_full + s)));
      }
    }
  } else {
    const int wg = (warp - 4) >> 2, q = warp & 3;
    const uint32_t first_tempty = in_first(smem_u32(tempty));
    uint32_t lt = 0;
    bool ok = true;
    Tile w;
    while (ok && walk.next(w)) {
      uint32_t v[4][32];  // one output of each of half of the tile's rows
      const int segments = segments_of(w);
      for (int s = 0; s < segments && ok; ++s, ++lt) {
        const uint32_t b = lt & 1u, use = lt >> 1;
        ok = wait_tmem(smem_u32(tfull + b), use & 1u, a.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t src = tmem + b * (uint32_t)kBQ + ((uint32_t)(32 * q) << 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = 64 * i + 32 * wg;  // chunks of 32 columns in turn
          if (c >= w.n) break;
          if (s == 0) {
            tmem_ld32(src + (uint32_t)c, v[i]);
          } else {
            uint32_t r[32];
            tmem_ld32(src + (uint32_t)c, r);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              v[i][j] = __float_as_uint(
                  __fadd_rn(__uint_as_float(v[i][j]), __uint_as_float(r[j])));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first(first_tempty + 8u * b);  // it may be overwritten
      }
      if (!ok) break;
      const bool none = w.kb0 == w.kb1;  // nothing was accumulated: zeros
      const int p = w.p0 + (int)rank * (kBP / 2) + 32 * q + lane;
      const int64_t plane = kCols ? (int64_t)w.g * a.Q : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = 64 * i + 32 * wg;
        if (c >= w.rows) break;
        if (none) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[i][j] = 0u;
        }
        if (p < a.P) store_rows<kCols>(a, v[i], (plane + w.q0 + c) * a.P + p, w.rows - c);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive_release();  // neither CTA leaves while the other uses its memory
  cluster_wait();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc2(tmem);
  }
}

// Row-major byte matrices [planes][rows][K], boxes of box_rows x 128 bytes.
bool make_map(CUtensorMap* map, const void* p, uint64_t K, uint64_t rows, uint64_t planes, int dims,
              uint32_t box_rows) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t d[3] = {K, rows, planes};
  const cuuint64_t st[2] = {K, K * rows};
  const cuuint32_t box[3] = {(cuuint32_t)kBK, box_rows, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)dims, const_cast<void*>(p), d, st,
                box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// p: [planes][P][inner], q: [q_rows][inner]; rows: the tokens or A's rows,
// which groups cut into at most `groups` ragged parts.
template <bool kCols>
int launch(const void* p, int64_t planes, const void* q, int64_t q_rows, int64_t inner,
           int64_t rows, int64_t groups, Args a, cudaStream_t stream) {
  a.status = device_status_ptr();
  if (!a.status) return QB_ECUDA;
  // Tiles of 224 rows; where those leave pairs of SMs without work, smaller
  // ones, down to 32 rows.
  const int64_t pairs = sm_count() / 2, np = (a.P + kBP - 1) / kBP;
  const auto tiles_of = [&](int bq) {
    return np * (kCols ? groups * ((rows + bq - 1) / bq) : rows / bq + groups);
  };
  a.bq = kBQ;
  while (a.bq > 32 && tiles_of(a.bq) < 2 * pairs) a.bq = a.bq == kBQ ? 128 : a.bq / 2;
  if (tiles_of(a.bq) > INT32_MAX) return QB_EOVERFLOW;
  a.np = (int)np;
  a.nq = (int)((rows + a.bq - 1) / a.bq);
  a.part = (int)(((rows + a.nq - 1) / a.nq + 15) / 16 * 16);
  CUtensorMap mp, mq32, mq8;
  if (!make_map(&mp, p, (uint64_t)inner, (uint64_t)a.P, (uint64_t)planes, 3, kBP / 2) ||
      !make_map(&mq32, q, (uint64_t)inner, (uint64_t)q_rows, 1, 2, 32) ||
      !make_map(&mq8, q, (uint64_t)inner, (uint64_t)q_rows, 1, 2, 8))
    return QB_ECUDA;
  static std::atomic<uint64_t> done{0};
  if (!smem_attribute(fp8_gemm_kernel<kCols>, kSmem, done)) return launch_status();
  const int64_t tiles = tiles_of(a.bq), grid = 2 * (pairs < tiles ? pairs : tiles);
  fp8_gemm_kernel<kCols><<<(unsigned)grid, kThreads, kSmem, stream>>>(mp, mq32, mq8, a);
  return launch_status();
}

}  // namespace

int launch_fp8_expert_gemm(const void* a, const uint8_t* a_scale, const void* b,
                           const uint8_t* b_scale, const int32_t* offsets, int G, int64_t M, int N,
                           int K, void* out, int out_dtype, cudaStream_t stream) {
  Args g{};
  g.sp = b_scale;
  g.sq = a_scale;
  g.offsets = offsets;
  g.out = out;
  g.tokens = M;
  g.P = N;
  g.kblocks = (K + kBK - 1) / kBK;
  g.G = G;
  g.pitch_p = g.pitch_q = (int)fp8_scale_pitch(K);
  g.p_blocks = (N + 127) / 128;
  g.f32 = out_dtype == QB_F32;
  return launch<false>(b, G, a, M, K, M, G < M ? G : M, g, stream);
}

int launch_fp8_expert_wgrad(const void* a_t, const uint8_t* a_scale, const void* b_t,
                            const uint8_t* b_scale, const int32_t* offsets, int G, int64_t width,
                            int N, int K, void* out, int out_dtype, int accumulate,
                            cudaStream_t stream) {
  Args g{};
  g.sp = b_scale;
  g.sq = a_scale;
  g.offsets = offsets;
  g.out = out;
  g.tokens = width;
  g.P = K;
  g.Q = N;
  g.kblocks = (int)(width / kBK);
  g.G = G;
  g.pitch_p = g.pitch_q = (int)fp8_scale_pitch(width);
  g.f32 = out_dtype == QB_F32;
  g.accumulate = accumulate;
  return launch<true>(b_t, 1, a_t, N, width, N, G, g, stream);
}

}  // namespace qb
