// qb_fp8.cu -- quantisers to e4m3 codes with one power-of-two scale for each
// 128 values, the operands of the experts' products (qb_fp8_gemm.cu).
//
//   e = the least whole number >= -127 with amax <= 448 * 2^e   (448: e4m3's largest)
//   code[i] = RN_e4m3(x[i] * 2^-e),   scale byte = e + 127 (e8m0)
//
// The product x * 2^-e is exact wherever its code is not zero or subnormal
// dust, so a code is one rounding of x.  amax is taken over the finite values;
// an infinity or NaN becomes the NaN code, and the product's row or column then
// shows it as a bf16 product would.  e comes from amax's bits: 448 = 1.75 * 2^8,
// so e = exponent - 8, and one more where the significand is above 1.75.
//
// What bounds all three is HBM (read x, write a byte per value): no value is
// read twice, every access is a whole 32-byte sector or more.
#include <cuda_bf16.h>

#include "qb_device.cuh"
#include "qb_internal.h"

namespace qb {
namespace {

constexpr uint32_t kInfBits = 0x7F800000u;

__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  const int b = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return b < 0 ? 0u : (uint32_t)b;
}
// 2^-e for e = byte - 127; byte is at most 247 here, so the result is normal
__device__ __forceinline__ float inverse_scale(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t finite_bits(uint32_t a) { return a < kInfBits ? a : 0u; }

__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t codes4(const float* v, float inv) {
  return codes2(__fmul_rn(v[0], inv), __fmul_rn(v[1], inv)) |
         codes2(__fmul_rn(v[2], inv), __fmul_rn(v[3], inv)) << 16;
}
// infinities to NaN, so that their code is NaN and not 448
__device__ __forceinline__ float loud(float v) {
  return abs_bits(v) >= kInfBits ? __uint_as_float(0x7FFFFFFFu) : v;
}

__device__ __forceinline__ void unpack8(uint4 u, float* v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
// 16 consecutive values
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float* v) {
  const uint4* q = reinterpret_cast<const uint4*>(p);
  const uint4 a = __ldg(q), b = __ldg(q + 1);
  unpack8(a, v);
  unpack8(b, v + 8);
}
__device__ __forceinline__ void load16(const float* p, float* v) {
  const float4* q = reinterpret_cast<const float4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 f = __ldg(q + i);
    v[4 * i] = f.x;
    v[4 * i + 1] = f.y;
    v[4 * i + 2] = f.z;
    v[4 * i + 3] = f.w;
  }
}
// 4 consecutive values
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* v) {
  const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
  v[0] = __uint_as_float(u.x << 16);
  v[1] = __uint_as_float(u.x & 0xFFFF0000u);
  v[2] = __uint_as_float(u.y << 16);
  v[3] = __uint_as_float(u.y & 0xFFFF0000u);
}
__device__ __forceinline__ void load4(const float* p, float* v) {
  const float4 f = __ldg(reinterpret_cast<const float4*>(p));
  v[0] = f.x;
  v[1] = f.y;
  v[2] = f.z;
  v[3] = f.w;
}

// ------------------------------------------------------------------ rows
// A warp codes 512 consecutive values of a row: 8 lanes of 16 values to a
// scale, four scales in the one 32-bit word that lane 0 writes.
template <typename T>
__global__ void __launch_bounds__(256)
    rows_kernel(const T* __restrict__ x, int64_t x_rows, int64_t ld,
                const int32_t* __restrict__ row_idx, int64_t M, int K, int words,
                uint8_t* __restrict__ q, uint32_t* __restrict__ scale) {
  const int lane = threadIdx.x & 31;
  const int64_t items = M * words;
  const int64_t step = (int64_t)gridDim.x * 8;
  for (int64_t it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); it < items; it += step) {
    const int64_t row = it / words;
    const int w = (int)(it - row * words);
    const int col = 512 * w + 16 * lane;
    int64_t src = row;
    if (row_idx) src = row_idx[row];
    const bool in = col < K;
    float v[16];
    if (in && src >= 0 && src < x_rows) {
      load16(x + src * ld + col, v);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, abs_bits(v[i]));
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (__any_sync(0xffffffffu, m >= kInfBits)) {
      m = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        m = max(m, finite_bits(abs_bits(v[i])));
        v[i] = loud(v[i]);
      }
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    }
    const uint32_t byte = scale_byte(m);
    const float inv = inverse_scale(byte);
    if (in)
      *reinterpret_cast<uint4*>(q + row * K + col) =
          make_uint4(codes4(v, inv), codes4(v + 4, inv), codes4(v + 8, inv), codes4(v + 12, inv));
    const uint32_t b0 = __shfl_sync(0xffffffffu, byte, 0), b1 = __shfl_sync(0xffffffffu, byte, 8),
                   b2 = __shfl_sync(0xffffffffu, byte, 16), b3 = __shfl_sync(0xffffffffu, byte, 24);
    if (lane == 0) scale[row * words + w] = b0 | b1 << 8 | b2 << 16 | b3 << 24;
  }
}

// ------------------------------------------------------------------ tiles
// 128 rows x 128 columns of x by 256 threads: warp w holds rows 16 w .. +15,
// lane l columns 4 l .. +3, so a row is one coalesced access of the warp and
// a thread's 16 values of a column are 16 bytes of the transposed codes.
struct TileRegs {
  float v[16][4];
};

// The transposed codes of a tile, [column][128 rows], in shared memory; the
// 16-byte chunks of a column are permuted by the column's number so that the
// lanes of a store (4 columns apart) meet different banks.
__device__ __forceinline__ uint4* transposed(unsigned char* sm, int col, int chunk) {
  return reinterpret_cast<uint4*>(sm + col * 128 + ((chunk ^ ((col >> 2) & 7)) << 4));
}

__device__ __forceinline__ void store_transposed(unsigned char* sm, const TileRegs& t,
                                                 const float (&inv)[4]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float w[4] = {t.v[4 * i][c], t.v[4 * i + 1][c], t.v[4 * i + 2][c], t.v[4 * i + 3][c]};
      u[i] = codes4(w, inv[c]);
    }
    *transposed(sm, 4 * lane + c, warp) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

__device__ __forceinline__ bool tile_has_nonfinite(const TileRegs& t) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) m = max(m, abs_bits(t.v[i][c]));
  return m >= kInfBits;
}

// Column maxima over this thread's 16 rows; non-finite values become NaN and
// do not count (`loudly`: there are any).
__device__ __forceinline__ void column_max(TileRegs& t, bool loudly, uint32_t (&m)[4]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) m[c] = 0;
  if (loudly) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        m[c] = max(m[c], finite_bits(abs_bits(t.v[i][c])));
        t.v[i][c] = loud(t.v[i][c]);
      }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) m[c] = max(m[c], abs_bits(t.v[i][c]));
  }
}

// Tokens in groups, scales along the tokens: x [rows, K] -> q_t [K, width],
// group g's tokens at columns from 128 * (blocks of the groups before g).
// A CTA codes four blocks of 128 tokens for 128 features, so that a feature's
// four scales are one 32-bit word.
template <typename T>
__global__ void __launch_bounds__(256)
    cols_kernel(const T* __restrict__ x, int64_t x_rows, int64_t ld,
                const int32_t* __restrict__ row_idx, const int32_t* __restrict__ offsets, int G,
                int64_t M, int K, int64_t width, int words, uint8_t* __restrict__ q_t,
                uint32_t* __restrict__ scale_t) {
  __shared__ __align__(16) unsigned char codes[128 * 128];
  __shared__ uint32_t part[8][128];
  __shared__ int pre[kMaxGroups + 1];
  __shared__ int64_t rows[128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  // running count of 128-token blocks per group, as the products count them
  for (int g = threadIdx.x; g < G; g += 256) {
    int64_t first = 0, end = M;
    if (offsets) {
      first = offsets[g];
      end = offsets[g + 1];
      first = first < 0 ? 0 : first > M ? M : first;
      end = end < first ? first : end > M ? M : end;
    }
    pre[g + 1] = (int)((end - first + 127) / 128);
  }
  __syncthreads();
  if (warp == 0) {
    int carry = 0;
    for (int g0 = 0; g0 < G; g0 += 32) {
      int v = g0 + lane < G ? pre[g0 + lane + 1] : 0;
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += u;
      }
      v = carry + v < (1 << 30) ? carry + v : 1 << 30;
      if (g0 + lane < G) pre[g0 + lane + 1] = v;
      carry = __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) pre[0] = 0;
  }
  __syncthreads();

  const int strips = (K + 127) / 128;
  const int strip = blockIdx.x % strips, run = blockIdx.x / strips;
  const int col = strip * 128 + 4 * lane;  // feature
  uint32_t word = 0;                            // threads 0-127: this feature's scales
  for (int i = 0; i < 4; ++i) {
    const int64_t b = (int64_t)run * 4 + i;
    if (b * 128 >= width) break;
    if (threadIdx.x < 128) {  // the source row of each of the block's tokens, or -1
      int64_t src = -1;
      if (b < pre[G]) {
        int lo = 0, hi = G - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (pre[mid] <= b) lo = mid; else hi = mid - 1;
        }
        int64_t first = 0, end = M;
        if (offsets) {
          first = offsets[lo];
          end = offsets[lo + 1];
          first = first < 0 ? 0 : first > M ? M : first;
          end = end < first ? first : end > M ? M : end;
        }
        const int64_t r = first + (b - pre[lo]) * 128 + threadIdx.x;
        if (r < end) src = row_idx ? row_idx[r] : r;
        if (src >= x_rows) src = -1;
      }
      rows[threadIdx.x] = src < 0 ? -1 : src;
    }
    __syncthreads();
    TileRegs t;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int64_t src = rows[16 * warp + r];
      if (src >= 0 && col < K) {
        load4(x + src * ld + col, t.v[r]);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) t.v[r][c] = 0.0f;
      }
    }
    uint32_t m[4];
    column_max(t, tile_has_nonfinite(t), m);
    *reinterpret_cast<uint4*>(&part[warp][4 * lane]) = make_uint4(m[0], m[1], m[2], m[3]);
    __syncthreads();
    float inv[4];
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const uint4 u = *reinterpret_cast<const uint4*>(&part[w][4 * lane]);
      m[0] = max(m[0], u.x);
      m[1] = max(m[1], u.y);
      m[2] = max(m[2], u.z);
      m[3] = max(m[3], u.w);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) inv[c] = inverse_scale(scale_byte(m[c]));
    if (threadIdx.x < 128) {
      uint32_t f = 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) f = max(f, part[w][threadIdx.x]);
      word |= scale_byte(f) << (8 * i);
    }
    store_transposed(codes, t, inv);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // 8 lanes write one feature's 128 bytes
      const int f = 32 * j + (threadIdx.x >> 3), chunk = threadIdx.x & 7;
      if (strip * 128 + f < K)
        *reinterpret_cast<uint4*>(q_t + (int64_t)(strip * 128 + f) * width + b * 128 +
                                  16 * chunk) = *transposed(codes, f, chunk);
    }
    __syncthreads();
  }
  const int f = strip * 128 + threadIdx.x;
  if (threadIdx.x < 128 && f < K) scale_t[(int64_t)f * words + run] = word;
}

// ------------------------------------------------------------------ 128 x 128 blocks
// Weights w [G, N, K]: one scale for each 128 x 128 block, the codes row-major
// and, where asked, transposed too (the same codes: a block's scale does not
// depend on the orientation).
template <typename T>
__global__ void __launch_bounds__(256)
    blocks_kernel(const T* __restrict__ x, int N, int K, int pitch, int pitch_t,
                  uint8_t* __restrict__ q, uint8_t* __restrict__ scale, uint8_t* __restrict__ q_t,
                  uint8_t* __restrict__ scale_t) {
  __shared__ __align__(16) unsigned char codes[128 * 128];
  __shared__ uint32_t part[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n_kb = (K + 127) / 128, n_nb = (N + 127) / 128;
  const int kb = blockIdx.x % n_kb, nb = blockIdx.x / n_kb % n_nb;
  const int64_t g = blockIdx.x / (n_kb * n_nb);
  const int col = kb * 128 + 4 * lane, row0 = nb * 128 + 16 * warp;
  const T* src = x + g * N * K;
  TileRegs t;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    if (row0 + r < N && col < K) {
      load4(src + (int64_t)(row0 + r) * K + col, t.v[r]);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) t.v[r][c] = 0.0f;
    }
  }
  uint32_t m[4];
  column_max(t, tile_has_nonfinite(t), m);
  uint32_t a = max(max(m[0], m[1]), max(m[2], m[3]));
  a = __reduce_max_sync(0xffffffffu, a);
  if (lane == 0) part[warp] = a;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) a = max(a, part[w]);
  const uint32_t byte = scale_byte(a);
  const float inv = inverse_scale(byte);
#pragma unroll
  for (int r = 0; r < 16; ++r)
    if (row0 + r < N && col < K)
      *reinterpret_cast<uint32_t*>(q + (g * N + row0 + r) * K + col) = codes4(t.v[r], inv);
  if (threadIdx.x == 0) {
    uint8_t* s = scale + (g * n_nb + nb) * pitch;
    s[kb] = (uint8_t)byte;
    if (kb == n_kb - 1)
      for (int i = n_kb; i < pitch; ++i) s[i] = 0;
    if (q_t) {
      uint8_t* st = scale_t + (g * n_kb + kb) * pitch_t;
      st[nb] = (uint8_t)byte;
      if (nb == n_nb - 1)
        for (int i = n_nb; i < pitch_t; ++i) st[i] = 0;
    }
  }
  if (!q_t) return;
  const float inv4[4] = {inv, inv, inv, inv};
  store_transposed(codes, t, inv4);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int f = 32 * j + (threadIdx.x >> 3), chunk = threadIdx.x & 7;
    const int k = kb * 128 + f, n = nb * 128 + 16 * chunk;
    if (k < K && n < N)
      *reinterpret_cast<uint4*>(q_t + (g * K + k) * N + n) = *transposed(codes, f, chunk);
  }
}

}  // namespace

int launch_fp8_rows(const void* x, int dtype, int64_t x_rows, int64_t ld, const int32_t* row_idx,
                    int64_t M, int K, uint8_t* q, uint8_t* scale, cudaStream_t stream) {
  const int words = (int)(fp8_scale_pitch(K) / 4);
  const int64_t items = M * words;
  int64_t grid = (items + 7) / 8;
  const int64_t most = 8 * (int64_t)sm_count();
  if (grid > most) grid = most;
  uint32_t* s = reinterpret_cast<uint32_t*>(scale);
  if (dtype == QB_F32)
    rows_kernel<float><<<(unsigned)grid, 256, 0, stream>>>(static_cast<const float*>(x), x_rows, ld,
                                                           row_idx, M, K, words, q, s);
  else
    rows_kernel<__nv_bfloat16><<<(unsigned)grid, 256, 0, stream>>>(
        static_cast<const __nv_bfloat16*>(x), x_rows, ld, row_idx, M, K, words, q, s);
  return launch_status();
}

int launch_fp8_cols(const void* x, int dtype, int64_t x_rows, int64_t ld, const int32_t* row_idx,
                    const int32_t* offsets, int G, int64_t M, int K, int64_t width, uint8_t* q_t,
                    uint8_t* scale_t, cudaStream_t stream) {
  const int words = (int)(fp8_scale_pitch(width) / 4);
  const unsigned grid = (unsigned)((K + 127) / 128) * (unsigned)words;
  uint32_t* s = reinterpret_cast<uint32_t*>(scale_t);
  if (dtype == QB_F32)
    cols_kernel<float><<<grid, 256, 0, stream>>>(static_cast<const float*>(x), x_rows, ld, row_idx,
                                                 offsets, G, M, K, width, words, q_t, s);
  else
    cols_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(static_cast<const __nv_bfloat16*>(x),
                                                         x_rows, ld, row_idx, offsets, G, M, K,
                                                         width, words, q_t, s);
  return launch_status();
}

int launch_fp8_blocks(const void* w, int dtype, int G, int N, int K, uint8_t* q, uint8_t* scale,
                      uint8_t* q_t, uint8_t* scale_t, cudaStream_t stream) {
  const unsigned grid = (unsigned)((K + 127) / 128) * (unsigned)((N + 127) / 128) * (unsigned)G;
  const int pitch = (int)fp8_scale_pitch(K), pitch_t = (int)fp8_scale_pitch(N);
  if (dtype == QB_F32)
    blocks_kernel<float><<<grid, 256, 0, stream>>>(static_cast<const float*>(w), N, K, pitch,
                                                   pitch_t, q, scale, q_t, scale_t);
  else
    blocks_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(static_cast<const __nv_bfloat16*>(w), N,
                                                           K, pitch, pitch_t, q, scale, q_t,
                                                           scale_t);
  return launch_status();
}

}  // namespace qb
