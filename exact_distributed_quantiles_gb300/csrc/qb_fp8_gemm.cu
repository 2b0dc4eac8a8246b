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
// accumulator, fp32 in tensor memory, is read once per tile.  The scale of a
// 128-value block serves the four MMAs of that block.
//
// One persistent CTA per SM walks tiles of 128 x BN outputs:
//   warp 0      TMA producer: 128 x 128 bytes of A and BN x 128 of B per stage
//               (128-byte swizzle);
//   warp 1      TMEM; one lane copies four K blocks' scales to tensor memory
//               at a time (tcgen05.cp) and issues four MMAs per K block;
//   warp 2      the scales' producer: one 32-bit word holds a row's scales of
//               four K blocks, laid out as tcgen05.cp wants them;
//   warps 4-11  two epilogue warpgroups, each half of the tile's columns.
// The rows of a group are known on the device only: each CTA sums the groups'
// tile counts itself, so the host never waits for the dispatch.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "qb_device.cuh"
#include "qb_internal.h"
#include "qb_tc.cuh"

namespace qb {
namespace {

constexpr int kBM = 128;
constexpr int kBK = 128;  // bytes of K per stage: one swizzle row
constexpr int kABytes = kBM * kBK;
constexpr int kSfStages = 4;
constexpr int kThreads = 12 * 32;
constexpr int kEpiThreads = 8 * 32;
constexpr int kStageRow = 80;  // staged output: 64 bytes of a row, 16 apart from the next
constexpr int kStageWarp = 32 * kStageRow;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kScaleCol = 256;  // accumulators below, scales from here

template <int BN>
struct Shape {
  static constexpr int stages = BN == 256 ? 4 : BN == 128 ? 6 : 8;
  static constexpr int b_bytes = BN * kBK;
  static constexpr int stage_bytes = kABytes + b_bytes;
  static constexpr int b_words = BN == 256 ? 8 : 4;  // scale words of B per lane
  static constexpr int sf_bytes = 512 + 128 * b_words;
  static constexpr int accumulators = BN == 256 ? 1 : 2;  // of BN columns, below kScaleCol
  static constexpr int smem = 1024 + stages * stage_bytes + kSfStages * sf_bytes +
                              8 * kStageWarp + 512 /*barriers*/ + 4 * (kMaxGroups + 4);
};

struct Args {
  const uint8_t* sa;
  const uint8_t* sb;
  const int32_t* offsets;  // nullptr: one group of all rows
  void* out;
  int64_t rows;   // rows of A (rows mode: tokens; cols mode: outputs n)
  int64_t tokens; // what offsets is clamped to
  int cols;       // outputs per row
  int kblocks;    // K blocks of every tile (rows mode), of the operands (cols mode)
  int G;
  int pitch_a, pitch_b;
  int b_blocks;   // rows mode: scale rows of B per group
  int f32, vec, accumulate;
  int* status;
};

__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc,
                                           uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X"
      " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// 32 rows x 16 bytes of shared memory -> 4 columns of tensor memory, the same
// in each of the four groups of 32 lanes.
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint32_t smem) {
  uint64_t d = 0;
  d |= (uint64_t)((smem & 0x3FFFFu) >> 4);
  d |= (uint64_t)(128 >> 4) << 32;  // 8 rows of 16 bytes to the next 8
  d |= (uint64_t)1 << 46;
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(d) : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(mbar)
      : "memory");
}

// Instruction descriptor, kind::mxf8f6f4: A and B e4m3 (format 0), K-major,
// N >> 3 at bits 17-22, scales e8m0 (bit 23), M >> 4 at bits 24-28; the byte of
// a scale word that serves this MMA at bits 29-30 (A) and 4-5 (B).
__device__ __forceinline__ uint32_t idesc_of(int BN, uint32_t byte) {
  return ((uint32_t)(BN >> 3) << 17) | (1u << 23) | ((uint32_t)(kBM >> 4) << 24) | (byte << 29) |
         (byte << 4);
}

// One tile of the walk.
struct Tile {
  int g;          // group
  int64_t row0;   // first row of A, and of the output within its plane
  int rows;       // rows that are stored
  int col0;       // first output column
  int kb0, kb1;   // K blocks
};

template <int BN, bool kCols>
__device__ __forceinline__ Tile tile_at(const Args& a, const int* pre, int64_t t) {
  Tile r;
  const int nt = (a.cols + BN - 1) / BN;
  const int64_t m = t / nt;
  r.col0 = (int)(t - m * nt) * BN;
  if (kCols) {
    const int mt = (int)((a.rows + kBM - 1) / kBM);
    r.g = (int)(m / mt);
    r.row0 = (m - (int64_t)r.g * mt) * kBM;
    const int64_t left = a.rows - r.row0;
    r.rows = left < kBM ? (int)left : kBM;
    r.kb0 = pre[r.g] < a.kblocks ? pre[r.g] : a.kblocks;
    r.kb1 = pre[r.g + 1] < a.kblocks ? pre[r.g + 1] : a.kblocks;
  } else {
    int lo = 0, hi = a.G - 1;  // the last group whose first tile is not after m
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= m) lo = mid; else hi = mid - 1;
    }
    r.g = lo;
    int64_t first = 0, end = a.tokens;
    if (a.offsets) {
      first = a.offsets[lo];
      end = a.offsets[lo + 1];
      first = first < 0 ? 0 : first > a.tokens ? a.tokens : first;
      end = end < first ? first : end > a.tokens ? a.tokens : end;
    }
    r.row0 = first + (m - pre[lo]) * kBM;
    const int64_t left = end - r.row0;
    r.rows = left < kBM ? (int)left : kBM;
    r.kb0 = 0;
    r.kb1 = a.kblocks;
  }
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

// Stores 32 rows x 32 columns of a warp (a lane holds its row's columns)
// through the warp's shared memory, so that a store instruction writes whole
// 64-byte pieces of rows.
__device__ __forceinline__ void store_chunk(const Args& a, const uint32_t (&v)[32],
                                            unsigned char* stage, int64_t at, int rows, int cols) {
  const int lane = threadIdx.x & 31;
  uint4* mine = reinterpret_cast<uint4*>(stage + lane * kStageRow);
  if (rows > 32) rows = 32;
  if (!a.f32) {
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + at;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        u[i] = bf16x2_rn(__uint_as_float(v[8 * j + 2 * i]), __uint_as_float(v[8 * j + 2 * i + 1]));
      mine[j] = make_uint4(u[0], u[1], u[2], u[3]);
    }
    __syncwarp();
    if (a.vec) {
      const int c = lane & 3;
#pragma unroll
      for (int r = lane >> 2; r < 32; r += 8)
        if (r < rows && 8 * c < cols)
          *reinterpret_cast<uint4*>(out + (int64_t)r * a.cols + 8 * c) =
              *reinterpret_cast<const uint4*>(stage + r * kStageRow + 16 * c);
    } else if (lane < cols) {
      for (int r = 0; r < rows; ++r)
        out[(int64_t)r * a.cols + lane] =
            *reinterpret_cast<const __nv_bfloat16*>(stage + r * kStageRow + 2 * lane);
    }
    __syncwarp();
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // 16 columns of fp32 at a time
    float* out = reinterpret_cast<float*>(a.out) + at + 16 * h;
    const int left = cols - 16 * h;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      mine[j] = make_uint4(v[16 * h + 4 * j], v[16 * h + 4 * j + 1], v[16 * h + 4 * j + 2],
                           v[16 * h + 4 * j + 3]);
    __syncwarp();
    if (a.vec) {
      const int c = lane & 3;
#pragma unroll
      for (int r = lane >> 2; r < 32; r += 8)
        if (r < rows && 4 * c < left) {
          float4* dst = reinterpret_cast<float4*>(out + (int64_t)r * a.cols + 4 * c);
          float4 f = *reinterpret_cast<const float4*>(stage + r * kStageRow + 16 * c);
          if (a.accumulate) {
            const float4 o = *dst;
            f = make_float4(o.x + f.x, o.y + f.y, o.z + f.z, o.w + f.w);
          }
          *dst = f;
        }
    } else {
      const int c = lane & 15;
      if (c < left)
        for (int r = lane >> 4; r < rows; r += 2) {
          float* dst = out + (int64_t)r * a.cols + c;
          const float f = *reinterpret_cast<const float*>(stage + r * kStageRow + 4 * c);
          *dst = a.accumulate ? *dst + f : f;
        }
    }
    __syncwarp();
  }
}

template <int BN, bool kCols>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap map_a,
                    const __grid_constant__ CUtensorMap map_a32,
                    const __grid_constant__ CUtensorMap map_b, const Args a) {
  constexpr int kStages = Shape<BN>::stages;
  constexpr int kBBytes = Shape<BN>::b_bytes;
  constexpr int kStageBytes = Shape<BN>::stage_bytes;
  constexpr int kSfBytes = Shape<BN>::sf_bytes;
  constexpr int kAcc = Shape<BN>::accumulators;

  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* sbase = smem_raw + (base - raw);
  unsigned char* sf = sbase + kStages * kStageBytes;
  unsigned char* stage_out = sf + kSfStages * kSfBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(stage_out + 8 * kStageWarp);
  uint64_t* empty = full + kStages;
  uint64_t* sf_full = empty + kStages;
  uint64_t* sf_empty = sf_full + kSfStages;
  uint64_t* tfull = sf_empty + kSfStages;
  uint64_t* tempty = tfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  int* pre = reinterpret_cast<int*>(reinterpret_cast<unsigned char*>(full) + 512);

  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int s = 0; s < kSfStages; ++s) {
      mbar_init(sf_full + s, 1);
      mbar_init(sf_empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull + b, 1);
      mbar_init(tempty + b, kEpiThreads);
    }
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), kTmemCols);
  // units of 128 rows (rows mode) or 128 columns (cols mode) of each group,
  // then their running sum: pre[g] = units of the groups before g
  for (int g = threadIdx.x; g < a.G; g += kThreads) {
    int64_t first = 0, end = a.tokens;
    if (a.offsets) {
      first = a.offsets[g];
      end = a.offsets[g + 1];
      first = first < 0 ? 0 : first > a.tokens ? a.tokens : first;
      end = end < first ? first : end > a.tokens ? a.tokens : end;
    }
    pre[g + 1] = (int)((end - first + 127) / 128);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {
    int carry = 0;
    for (int g0 = 0; g0 < a.G; g0 += 32) {
      int v = g0 + lane < a.G ? pre[g0 + lane + 1] : 0;
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += u;
      }
      // offsets that do not ascend could add up without end: the sum stops at 2^30
      v = carry + v < (1 << 30) ? carry + v : 1 << 30;
      if (g0 + lane < a.G) pre[g0 + lane + 1] = v;
      carry = __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) pre[0] = 0;
  }
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  const int64_t col_tiles = (a.cols + BN - 1) / BN;
  const int64_t n_tiles =
      kCols ? (int64_t)a.G * ((a.rows + kBM - 1) / kBM) * col_tiles : (int64_t)pre[a.G] * col_tiles;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t gk = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; t < n_tiles && ok; t += gridDim.x) {
        const Tile w = tile_at<BN, kCols>(a, pre, t);
        // a tile of few rows reads only the boxes of 32 rows that hold them;
        // the rest of the stage keeps old codes, whose products are not stored
        const int boxes = (w.rows + 31) >> 5;
        for (int kb = w.kb0; kb < w.kb1; ++kb, ++gk) {
          const int s = (int)(gk % kStages);
          if (gk >= (uint32_t)kStages &&
              !mbar_wait_bounded(empty + s, (gk / kStages - 1) & 1u, a.status)) {
            ok = false;
            break;
          }
          const uint32_t sa = base + (uint32_t)(s * kStageBytes), bar = smem_u32(full + s);
          mbar_arrive_expect_tx(full + s, (uint32_t)(boxes * 32 * kBK + kBBytes));
          if (boxes == 4) {
            tma_load_2d(sa, &map_a, kb * kBK, (int)w.row0, bar);
          } else {
            for (int i = 0; i < boxes; ++i)
              tma_load_2d(sa + 32u * kBK * i, &map_a32, kb * kBK, (int)w.row0 + 32 * i, bar);
          }
          tma_load_3d(sa + kABytes, &map_b, kb * kBK, w.col0, kCols ? 0 : w.g, bar);
        }
      }
      if (!ok) {  // leave no copy in flight
        const uint32_t back = gk < (uint32_t)kStages ? gk : (uint32_t)kStages;
        for (uint32_t i = gk - back; i < gk; ++i)
          mbar_wait_bounded(full + i % kStages, (i / kStages) & 1u, a.status);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t gk = 0, gs = 0, lt = 0;
      const uint32_t sfa = tmem + kScaleCol, sfb = sfa + 4;
      bool ok = true;
      for (int64_t t = blockIdx.x; t < n_tiles && ok; t += gridDim.x) {
        const Tile w = tile_at<BN, kCols>(a, pre, t);
        const int segments = segments_of(w);
        int kb = w.kb0;
        for (int seg = 0; seg < segments && ok; ++seg, ++lt) {
          const uint32_t b = lt % kAcc, use = lt / kAcc;
          if (use >= 1 && !mbar_wait_bounded(tempty + b, (use - 1) & 1u, a.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + b * (uint32_t)BN;
          const int end = w.kb1 - kb < kSegment ? w.kb1 : kb + kSegment;
          for (uint32_t first = 0; kb < end; ++kb, ++gk, first = 1) {
            if (kb == w.kb0 || (kb & 3) == 0) {
              const int s = (int)(gs % kSfStages);
              if (!mbar_wait_bounded(sf_full + s, (gs / kSfStages) & 1u, a.status)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint32_t src = smem_u32(sf + s * kSfBytes);
              copy_scales(sfa, src);
              copy_scales(sfb, src + 512);
              if (BN == 256) copy_scales(sfb + 4, src + 1024);
              tc_commit(smem_u32(sf_empty + s));
              ++gs;
            }
            const int s = (int)(gk % kStages);
            if (!mbar_wait_bounded(full + s, (gk / kStages) & 1u, a.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa = base + (uint32_t)(s * kStageBytes);
            const uint32_t idesc = idesc_of(BN, (uint32_t)(kb & 3));
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // 32 values of K, 32 bytes along the row
              mma_scaled(d, smem_desc_sw128(sa + 32u * kk),
                         smem_desc_sw128(sa + kABytes + 32u * kk), idesc, sfa, sfb,
                         kk > 0 ? 1u : first);
            tc_commit(smem_u32(empty + s));
          }
          if (ok) tc_commit(smem_u32(tfull + b));
        }
      }
    }
  } else if (warp == 2) {
    uint32_t gs = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; t < n_tiles && ok; t += gridDim.x) {
      const Tile w = tile_at<BN, kCols>(a, pre, t);
      for (int c = w.kb0 >> 2; w.kb0 < w.kb1 && 4 * c < w.kb1; ++c, ++gs) {
        // lane l holds rows l, l + 32, l + 64 and l + 96 of each 128
        constexpr int kWordsB = Shape<BN>::b_words;
        uint32_t va[4], vb[kWordsB];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = lane + 32 * j;
          va[j] = r < w.rows ? __ldg(reinterpret_cast<const uint32_t*>(
                                   a.sa + (w.row0 + r) * a.pitch_a + 4 * c))
                             : 0u;
        }
#pragma unroll
        for (int j = 0; j < kWordsB; ++j) {
          const int n = w.col0 + (kCols ? lane + 32 * j : 32 * j);
          const int64_t row = kCols ? n : (int64_t)w.g * a.b_blocks + n / 128;
          vb[j] = n < a.cols && 32 * j < BN
                      ? __ldg(reinterpret_cast<const uint32_t*>(a.sb + row * a.pitch_b + 4 * c))
                      : 0u;
        }
        const int s = (int)(gs % kSfStages);
        if (gs >= (uint32_t)kSfStages &&
            !mbar_wait_bounded(sf_empty + s, (gs / kSfStages - 1) & 1u, a.status))
          ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint4* dst = reinterpret_cast<uint4*>(sf + s * kSfBytes) + lane;
        dst[0] = make_uint4(va[0], va[1], va[2], va[3]);
#pragma unroll
        for (int j = 0; j < kWordsB; j += 4)
          dst[32 + 8 * j] = make_uint4(vb[j], vb[j + 1], vb[j + 2], vb[j + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(sf_full + s);
      }
    }
  } else if (warp >= 4) {
    const int wg = (warp - 4) >> 2, q = warp & 3;
    unsigned char* mine = stage_out + (warp - 4) * kStageWarp;
    uint32_t lt = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; t < n_tiles && ok; t += gridDim.x) {
      const Tile w = tile_at<BN, kCols>(a, pre, t);
      uint32_t v[BN / 64][32];  // this thread's row, half of the tile's columns
      const int segments = segments_of(w);
      for (int s = 0; s < segments && ok; ++s, ++lt) {
        const uint32_t b = lt % kAcc, use = lt / kAcc;
        ok = mbar_wait_bounded(tfull + b, use & 1u, a.status);
        ok = __all_sync(0xffffffffu, ok);  // tcgen05.ld is warp-collective
        if (!ok) break;
        tc_fence_after();
        const uint32_t src =
            tmem + b * (uint32_t)BN + (uint32_t)(wg * (BN / 2)) + ((uint32_t)(32 * q) << 16);
        if (s == 0) {
#pragma unroll
          for (int i = 0; i < BN / 64; ++i) tmem_ld32_nowait(src + 32u * i, v[i]);
#pragma unroll
          for (int i = 0; i < BN / 64; ++i) tmem_wait_ld(v[i]);
        } else {
#pragma unroll
          for (int i = 0; i < BN / 64; ++i) {
            uint32_t r[32];
            tmem_ld32(src + 32u * i, r);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              v[i][j] = __float_as_uint(
                  __fadd_rn(__uint_as_float(v[i][j]), __uint_as_float(r[j])));
          }
        }
        tc_fence_before();
        mbar_arrive(tempty + b);  // the accumulator may be overwritten
      }
      if (!ok) break;
      const bool none = w.kb0 == w.kb1;  // nothing was accumulated: zeros
      const int rows = w.rows - 32 * q;
      const int64_t plane = kCols ? (int64_t)w.g * a.rows : 0;
      const int64_t at = (plane + w.row0 + 32 * q) * a.cols;
#pragma unroll
      for (int i = 0; i < BN / 64; ++i) {
        const int col = w.col0 + wg * (BN / 2) + 32 * i;
        if (none) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[i][j] = 0u;
        }
        if (rows > 0 && col < a.cols) store_chunk(a, v[i], mine, at + col, rows, a.cols - col);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
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

template <int BN, bool kCols>
int launch_bn(const void* pa, const void* pb, int64_t a_rows, int64_t b_rows, int64_t b_planes,
              int64_t inner, int64_t tiles, const Args& a, cudaStream_t stream) {
  CUtensorMap ma, ma32, mb;
  if (!make_map(&ma, pa, (uint64_t)inner, (uint64_t)a_rows, 1, 2, kBM) ||
      !make_map(&ma32, pa, (uint64_t)inner, (uint64_t)a_rows, 1, 2, 32) ||
      !make_map(&mb, pb, (uint64_t)inner, (uint64_t)b_rows, (uint64_t)b_planes, 3, BN))
    return QB_ECUDA;
  static std::atomic<uint64_t> done{0};
  if (!smem_attribute(fp8_gemm_kernel<BN, kCols>, Shape<BN>::smem, done)) return launch_status();
  int64_t grid = sm_count();
  if (grid > tiles) grid = tiles;
  fp8_gemm_kernel<BN, kCols><<<(unsigned)grid, kThreads, Shape<BN>::smem, stream>>>(ma, ma32, mb, a);
  return launch_status();
}

// The tile's width: 256 columns feed the tensor cores best; where that leaves
// SMs without a tile, narrower ones spread the weights over more of them.
int pick_bn(int64_t row_tiles, int cols) {
  const int64_t sms = sm_count();
  if (row_tiles * ((cols + 255) / 256) >= 2 * sms) return 256;
  if (row_tiles * ((cols + 127) / 128) >= 2 * sms) return 128;
  return 64;
}

template <bool kCols>
int launch_any(const void* pa, const void* pb, int64_t a_rows, int64_t b_rows, int64_t b_planes,
               int64_t inner, int64_t row_tiles, Args a, cudaStream_t stream) {
  a.status = device_status_ptr();
  if (!a.status) return QB_ECUDA;
  a.vec = a.cols % (a.f32 ? 4 : 8) == 0;
  const int bn = pick_bn(row_tiles, a.cols);
  const int64_t tiles = row_tiles * ((a.cols + bn - 1) / bn);
  if (bn == 256)
    return launch_bn<256, kCols>(pa, pb, a_rows, b_rows, b_planes, inner, tiles, a, stream);
  if (bn == 128)
    return launch_bn<128, kCols>(pa, pb, a_rows, b_rows, b_planes, inner, tiles, a, stream);
  return launch_bn<64, kCols>(pa, pb, a_rows, b_rows, b_planes, inner, tiles, a, stream);
}

}  // namespace

int launch_fp8_expert_gemm(const void* a, const uint8_t* a_scale, const void* b,
                           const uint8_t* b_scale, const int32_t* offsets, int G, int64_t M, int N,
                           int K, void* out, int out_dtype, cudaStream_t stream) {
  Args g{};
  g.sa = a_scale;
  g.sb = b_scale;
  g.offsets = offsets;
  g.out = out;
  g.rows = g.tokens = M;
  g.cols = N;
  g.kblocks = (K + kBK - 1) / kBK;
  g.G = G;
  g.pitch_a = g.pitch_b = (int)fp8_scale_pitch(K);
  g.b_blocks = (N + 127) / 128;
  g.f32 = out_dtype == QB_F32;
  // at most one ragged tile per group that has a row
  const int64_t row_tiles = M / kBM + (G < M ? G : M);
  return launch_any<false>(a, b, M, N, G, K, row_tiles, g, stream);
}

int launch_fp8_expert_wgrad(const void* a_t, const uint8_t* a_scale, const void* b_t,
                            const uint8_t* b_scale, const int32_t* offsets, int G, int64_t width,
                            int N, int K, void* out, int out_dtype, int accumulate,
                            cudaStream_t stream) {
  Args g{};
  g.sa = a_scale;
  g.sb = b_scale;
  g.offsets = offsets;
  g.out = out;
  g.rows = N;
  g.tokens = width;
  g.cols = K;
  g.kblocks = (int)(width / kBK);
  g.G = G;
  g.pitch_a = g.pitch_b = (int)fp8_scale_pitch(width);
  g.f32 = out_dtype == QB_F32;
  g.accumulate = accumulate;
  const int64_t row_tiles = (int64_t)G * ((N + kBM - 1) / kBM);
  return launch_any<true>(a_t, b_t, N, K, 1, width, row_tiles, g, stream);
}

}  // namespace qb
