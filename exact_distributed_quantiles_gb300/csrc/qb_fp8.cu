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
// HBM is the floor of all three (read x, write a byte per value): no output
// needs a value twice, every access is a whole 32-byte sector or more.  A row
// that the indexes name several times is fetched and coded for each of them.
// Measured, bf16: 64 x 1024 x 2048 weights in both orientations 86 us (6.2
// TB/s); 196608 rows of 2048 gathered from 32768, 127 us (5.5 TB/s of traffic:
// the source, 134 MB, does not quite fit in L2 and 335 MB are read; integer
// unit 67% busy); token-major 65536 x 2048, 73 us.
#include <cuda_bf16.h>

#include "qb_device.cuh"
#include "qb_groups.cuh"
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

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Codes of two pairs of values, each pair multiplied by its own pair of scales.
__device__ __forceinline__ uint32_t codes4(f2_t a, f2_t b, f2_t inv_a, f2_t inv_b) {
  float lo, hi;
  uint16_t ra, rb;
  f2_unpack(f2_mul(a, inv_a), lo, hi);
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(ra) : "f"(hi), "f"(lo));
  f2_unpack(f2_mul(b, inv_b), lo, hi);
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(rb) : "f"(hi), "f"(lo));
  return (uint32_t)ra | (uint32_t)rb << 16;
}

// Four consecutive values as they come from memory.  The largest magnitude is
// taken on the bits (they order like the magnitudes), for bf16 two at a time.
template <typename T>
struct Four;

template <>
struct Four<__nv_bfloat16> {
  uint2 u;
  struct Max {  // magnitudes' bits of four columns
    uint32_t a, b;
    __device__ __forceinline__ void add(const Max& o) {
      a = max_u16x2(a, o.a);
      b = max_u16x2(b, o.b);
    }
    __device__ __forceinline__ Max shuffled(int d) const {
      return Max{__shfl_xor_sync(0xffffffffu, a, d), __shfl_xor_sync(0xffffffffu, b, d)};
    }
    __device__ __forceinline__ bool nonfinite() const {
      const uint32_t m = max_u16x2(a, b);
      return (m & 0xFFFFu) >= 0x7F80u || m >= 0x7F800000u;
    }
    __device__ __forceinline__ void columns(uint32_t (&m)[4]) const {  // as fp32 bits
      m[0] = a << 16;
      m[1] = a & 0xFFFF0000u;
      m[2] = b << 16;
      m[3] = b & 0xFFFF0000u;
    }
    __device__ __forceinline__ uint32_t all() const {
      const uint32_t m = max_u16x2(a, b);
      return max(m << 16, m & 0xFFFF0000u);
    }
  };
  __device__ __forceinline__ void zero() { u = make_uint2(0u, 0u); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    u = __ldg(reinterpret_cast<const uint2*>(p));
  }
  __device__ __forceinline__ void max_into(Max& m) const {
    m.a = max_u16x2(m.a, u.x & 0x7FFF7FFFu);
    m.b = max_u16x2(m.b, u.y & 0x7FFF7FFFu);
  }
  // The same by the half-precision unit, which keeps NaN: less work for the
  // integer unit, on which the conversions run (rows 135 -> 131 us and
  // token-major codes 77 -> 75 us at the sizes below; the weights' kernel, with
  // its byte permutes after the loads, is faster with the integer form, 85
  // against 89 us).
  __device__ __forceinline__ void max_into_h(Max& m) const {
    uint32_t x, y;
    asm("abs.bf16x2 %0, %1;" : "=r"(x) : "r"(u.x));
    asm("abs.bf16x2 %0, %1;" : "=r"(y) : "r"(u.y));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m.a) : "r"(m.a), "r"(x));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m.b) : "r"(m.b), "r"(y));
  }
  // infinities become NaN; the finite magnitudes alone count
  __device__ __forceinline__ static uint32_t loud2(uint32_t w, uint32_t& m) {
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
      const uint32_t b = (w >> h) & 0x7FFFu;
      if (b >= 0x7F80u)
        w |= 0x7Fu << h;
      else
        m = max_u16x2(m, b << h);
    }
    return w;
  }
  __device__ __forceinline__ void loud(Max& m) {
    u.x = loud2(u.x, m.a);
    u.y = loud2(u.y, m.b);
  }
  __device__ __forceinline__ uint32_t codes(f2_t inv01, f2_t inv23) const {
    return codes4(f2_pack(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u)),
                  f2_pack(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u)), inv01,
                  inv23);
  }
};

template <>
struct Four<float> {
  float4 f;
  struct Max {
    uint32_t m0, m1, m2, m3;
    __device__ __forceinline__ void add(const Max& o) {
      m0 = max(m0, o.m0);
      m1 = max(m1, o.m1);
      m2 = max(m2, o.m2);
      m3 = max(m3, o.m3);
    }
    __device__ __forceinline__ Max shuffled(int d) const {
      return Max{__shfl_xor_sync(0xffffffffu, m0, d), __shfl_xor_sync(0xffffffffu, m1, d),
                 __shfl_xor_sync(0xffffffffu, m2, d), __shfl_xor_sync(0xffffffffu, m3, d)};
    }
    __device__ __forceinline__ bool nonfinite() const { return all() >= kInfBits; }
    __device__ __forceinline__ void columns(uint32_t (&m)[4]) const {
      m[0] = m0;
      m[1] = m1;
      m[2] = m2;
      m[3] = m3;
    }
    __device__ __forceinline__ uint32_t all() const { return max(max(m0, m1), max(m2, m3)); }
  };
  __device__ __forceinline__ void zero() { f = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ void load(const float* p) {
    f = __ldg(reinterpret_cast<const float4*>(p));
  }
  __device__ __forceinline__ void max_into(Max& m) const {
    m.m0 = max(m.m0, abs_bits(f.x));
    m.m1 = max(m.m1, abs_bits(f.y));
    m.m2 = max(m.m2, abs_bits(f.z));
    m.m3 = max(m.m3, abs_bits(f.w));
  }
  __device__ __forceinline__ void max_into_h(Max& m) const { max_into(m); }
  __device__ __forceinline__ static void loud1(float& v, uint32_t& m) {
    const uint32_t b = abs_bits(v);
    if (b >= kInfBits)
      v = __uint_as_float(0x7FFFFFFFu);
    else
      m = max(m, b);
  }
  __device__ __forceinline__ void loud(Max& m) {
    loud1(f.x, m.m0);
    loud1(f.y, m.m1);
    loud1(f.z, m.m2);
    loud1(f.w, m.m3);
  }
  __device__ __forceinline__ uint32_t codes(f2_t inv01, f2_t inv23) const {
    return codes4(f2_pack(f.x, f.y), f2_pack(f.z, f.w), inv01, inv23);
  }
};

// 16 consecutive values
template <typename T>
__device__ __forceinline__ void load16(const T* p, Four<T> (&v)[4]);
template <>
__device__ __forceinline__ void load16(const __nv_bfloat16* p, Four<__nv_bfloat16> (&v)[4]) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
  const uint4 b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
  v[0].u = make_uint2(a.x, a.y);
  v[1].u = make_uint2(a.z, a.w);
  v[2].u = make_uint2(b.x, b.y);
  v[3].u = make_uint2(b.z, b.w);
}
template <>
__device__ __forceinline__ void load16(const float* p, Four<float> (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i].load(p + 4 * i);
}

// ------------------------------------------------------------------ rows
// A warp codes 512 consecutive values of a row: 8 lanes of 16 values to a
// scale, four scales in the one 32-bit word that lane 0 writes.  Several rows
// of a warp are in flight together, their row numbers read ahead of the rows.
template <typename T>
struct RowsShape {
  static constexpr int in_flight = sizeof(T) == 2 ? 3 : 2;  // rows of a warp
  static constexpr int ctas = sizeof(T) == 2 ? 5 : 4;       // to an SM
};

template <typename T>
__global__ void __launch_bounds__(256, RowsShape<T>::ctas)
    rows_kernel(const T* __restrict__ x, int64_t x_rows, int64_t ld,
                const int32_t* __restrict__ row_idx, int64_t M, int K, int words,
                uint8_t* __restrict__ q, uint32_t* __restrict__ scale) {
  constexpr int U = RowsShape<T>::in_flight;
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * 8;
  const int w = blockIdx.y, col = 512 * w + 16 * lane;
  const bool in = col < K;
  for (int64_t r0 = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); r0 < M; r0 += U * step) {
    int64_t src[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t row = r0 + i * step;
      src[i] = row < M ? (row_idx ? __ldg(row_idx + row) : row) : -1;
    }
    Four<T> v[U][4];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (in && src[i] >= 0 && src[i] < x_rows) {
        load16(x + src[i] * ld + col, v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j].zero();
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t row = r0 + i * step;
      if (row >= M) break;
      typename Four<T>::Max mx{};
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j].max_into_h(mx);
      uint32_t m = mx.all();
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
      if (__any_sync(0xffffffffu, m >= kInfBits)) {
        typename Four<T>::Max fin{};
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j].loud(fin);
        m = fin.all();
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
      }
      const uint32_t byte = scale_byte(m);
      const f2_t inv = f2_splat(inverse_scale(byte));
      if (in)
        *reinterpret_cast<uint4*>(q + row * K + col) =
            make_uint4(v[i][0].codes(inv, inv), v[i][1].codes(inv, inv), v[i][2].codes(inv, inv),
                       v[i][3].codes(inv, inv));
      uint32_t word = byte << (lane & 24);
      word |= __shfl_xor_sync(0xffffffffu, word, 8);
      word |= __shfl_xor_sync(0xffffffffu, word, 16);
      if (lane == 0) scale[row * words + w] = word;
    }
  }
}

// ------------------------------------------------------------------ tiles
// 16 rows x 4 columns of a thread, for the two kernels that transpose.

// Column maxima of a thread's 16 rows.
template <typename T, bool kHalf>
__device__ __forceinline__ typename Four<T>::Max column_max(Four<T> (&v)[16]) {
  typename Four<T>::Max m{};
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    if (kHalf)
      v[r].max_into_h(m);
    else
      v[r].max_into(m);
  }
  if (m.nonfinite()) {
    m = typename Four<T>::Max{};
#pragma unroll
    for (int r = 0; r < 16; ++r) v[r].loud(m);
  }
  return m;
}

// Codes r[i] of four columns in rows i = 0..15 -> c[j], the 16 codes of column
// j: 4 x 4 bytes at a time by byte permutes.
__device__ __forceinline__ void transpose16(const uint32_t (&r)[16], uint4 (&c)[4]) {
  uint32_t o[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t t0 = prmt(r[4 * i], r[4 * i + 1], 0x5140u);
    const uint32_t t1 = prmt(r[4 * i + 2], r[4 * i + 3], 0x5140u);
    const uint32_t t2 = prmt(r[4 * i], r[4 * i + 1], 0x7362u);
    const uint32_t t3 = prmt(r[4 * i + 2], r[4 * i + 3], 0x7362u);
    o[0][i] = prmt(t0, t1, 0x5410u);
    o[1][i] = prmt(t0, t1, 0x7632u);
    o[2][i] = prmt(t2, t3, 0x5410u);
    o[3][i] = prmt(t2, t3, 0x7632u);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) c[j] = make_uint4(o[j][0], o[j][1], o[j][2], o[j][3]);
}

// The transposed codes of a tile, [column][128 rows], in shared memory; the
// 16-byte chunks of a column are permuted by the column's number so that the
// lanes of a store (4 columns apart) meet different banks.
__device__ __forceinline__ uint4* transposed(unsigned char* sm, int col, int chunk) {
  return reinterpret_cast<uint4*>(sm + col * 128 + ((chunk ^ ((col >> 2) & 7)) << 4));
}

// r[i]: the codes of this thread's four columns in row i.
__device__ __forceinline__ void store_transposed(unsigned char* sm, const uint32_t (&r)[16]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint4 c[4];
  transpose16(r, c);
#pragma unroll
  for (int j = 0; j < 4; ++j) *transposed(sm, 4 * lane + j, warp) = c[j];
}

// ------------------------------------------------------------------ token-major
// Tokens in groups, scales along the tokens: x [rows, K] -> q_t [K, width],
// group g's tokens at columns from 128 * (blocks of the groups before g).
//
// A warp codes 128 tokens x 32 features (16 of fp32) by itself: lane l holds
// tokens 16 (l / 4) .. +15 of the 16 bytes l % 4 of a row's 64, so that a
// feature's maximum takes three shuffles, a lane's 16 codes of a feature are 16
// consecutive bytes and a store instruction writes the 128 bytes of four
// features.  Nothing
// passes between warps: with the amax and the transpose through shared memory
// and barriers the same work took 76 us at 65536 x 2048 gathered bf16 rows,
// this 73 (219 MB cannot be avoided: 33 us; the integer unit, the L1's data
// path and the issue slots are each 55% busy).  The warps of a CTA take
// the same tokens, which makes their 64-byte pieces of a row whole lines.  A
// CTA walks a run of consecutive blocks of one strip of features after another.  A feature's scales of four blocks make one 32-bit word; words that
// the run covers in part are written by bytes.
template <typename T>
struct ColsShape {
  static constexpr int quads = sizeof(T) == 2 ? 2 : 1;  // of four features of a lane
  static constexpr int warps = 4;
  static constexpr int features = warps * 16 * quads;
  static constexpr int ctas = 5;  // to an SM
};

__device__ __forceinline__ void load_quads(const __nv_bfloat16* p, Four<__nv_bfloat16> (&v)[2]) {
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  v[0].u = make_uint2(u.x, u.y);
  v[1].u = make_uint2(u.z, u.w);
}
__device__ __forceinline__ void load_quads(const float* p, Four<float> (&v)[1]) { v[0].load(p); }

template <typename T>
__global__ void __launch_bounds__(ColsShape<T>::warps * 32, ColsShape<T>::ctas)
    cols_kernel(const T* __restrict__ x, int64_t x_rows, int64_t ld,
                const int32_t* __restrict__ row_idx, const int32_t* __restrict__ offsets, int G,
                int64_t M, int K, int64_t width, int words, int64_t run,
                uint8_t* __restrict__ q_t, uint8_t* __restrict__ scale_t) {
  __shared__ int pre[kMaxGroups + 1], start[kMaxGroups + 1];
  constexpr int kQuads = ColsShape<T>::quads, kStrip = ColsShape<T>::features;
  __shared__ __align__(16) int rows[ColsShape<T>::warps][128];  // a warp's source rows, -1: zeros
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blocks = (int)(width / 128);
  const int64_t units = (int64_t)((K + kStrip - 1) / kStrip) * blocks;
  const int64_t u0 = blockIdx.x * run;
  const int64_t u1 = u0 + run < units ? u0 + run : units;
  count_units(offsets, G, (int)M, 128, start, pre);
  __syncthreads();

  // four source rows of a lane: tokens 4 lane .. +3 of block b
  const auto look_up = [&](int b, int (&src)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) src[i] = -1;
    if (b >= pre[G]) return;
    const int g = group_of(pre, G, b), end = start[g + 1];
    const int r = start[g] + (b - pre[g]) * 128 + 4 * lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (r + i < end) src[i] = row_idx ? __ldg(row_idx + r + i) : r + i;
      if (src[i] >= x_rows) src[i] = -1;
    }
  };
  int strip = (int)(u0 / blocks), b = (int)(u0 - (int64_t)strip * blocks);
  int src[4];
  if (u0 < u1) look_up(b, src);

  uint32_t word[kQuads][4] = {}, covered = 0;  // lanes 0-3: scales of their features
  for (int64_t u = u0; u < u1; ++u) {
    const int col = strip * kStrip + (16 * warp + 4 * (lane & 3)) * kQuads;
    *reinterpret_cast<int4*>(&rows[warp][4 * lane]) = make_int4(src[0], src[1], src[2], src[3]);
    __syncwarp();
    Four<T> v[16][kQuads];
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      const int4 s = *reinterpret_cast<const int4*>(&rows[warp][16 * (lane >> 2) + r]);
      const int at[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (at[i] >= 0 && col < K) {
          load_quads(x + at[i] * ld + col, v[r + i]);
        } else {
#pragma unroll
          for (int h = 0; h < kQuads; ++h) v[r + i][h].zero();
        }
      }
    }
    __syncwarp();
    const int next_b = b + 1 < blocks ? b + 1 : 0;
    if (u + 1 < u1) look_up(next_b, src);
    covered |= 1u << (b & 3);
    if (b == blocks - 1) covered |= 0xEu << (b & 3) & 0xFu;  // zeros behind the last block
    const bool flush = (b & 3) == 3 || b == blocks - 1 || u + 1 == u1;
#pragma unroll
    for (int h = 0; h < kQuads; ++h) {
      Four<T> w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = v[i][h];
      typename Four<T>::Max m = column_max<T, true>(w);
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) m.add(m.shuffled(d));
      uint32_t c[4];
      m.columns(c);
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = scale_byte(c[i]);
      const f2_t inv01 = f2_pack(inverse_scale(c[0]), inverse_scale(c[1]));
      const f2_t inv23 = f2_pack(inverse_scale(c[2]), inverse_scale(c[3]));
      uint32_t r[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) r[i] = w[i].codes(inv01, inv23);
      uint4 o[4];
      transpose16(r, o);
      const int f = col + 4 * h;
      if (col < K) {
        uint8_t* dst = q_t + (int64_t)f * width + (int64_t)b * 128 + 16 * (lane >> 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(dst + j * width) = o[j];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        word[h][i] |= c[i] << (8 * (b & 3));
        if (flush) {
          if (lane < 4 && col < K) {
            uint8_t* s = scale_t + ((int64_t)(f + i) * words + (b >> 2)) * 4;
            if (covered == 0xFu) {
              *reinterpret_cast<uint32_t*>(s) = word[h][i];
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (covered >> j & 1u) s[j] = (uint8_t)(word[h][i] >> (8 * j));
            }
          }
          word[h][i] = 0;
        }
      }
    }
    if (flush) covered = 0;
    b = next_b;
    if (b == 0) ++strip;
  }
}

// ------------------------------------------------------------------ 128 x 128 blocks
// Weights w [G, N, K]: one scale for each 128 x 128 block, the codes row-major
// and, where asked, transposed too (the same codes: a block's scale does not
// depend on the orientation).  256 threads: warp w holds rows 16 w .. +15, lane
// l columns 4 l .. +3, so a row is one coalesced access of the warp and a
// thread's 16 values of a column are 16 bytes of the transposed codes.
template <typename T>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 2)
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
  const T* src = x + (g * N + row0) * K + col;
  Four<T> v[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    if (row0 + r < N && col < K)
      v[r].load(src + (int64_t)r * K);
    else
      v[r].zero();
  }
  uint32_t a = __reduce_max_sync(0xffffffffu, column_max<T, false>(v).all());
  if (lane == 0) part[warp] = a;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) a = max(a, part[w]);
  const uint32_t byte = scale_byte(a);
  const f2_t inv = f2_splat(inverse_scale(byte));
  uint32_t c[16];
  uint8_t* dst = q + (g * N + row0) * K + col;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    c[r] = v[r].codes(inv, inv);
    if (row0 + r < N && col < K) *reinterpret_cast<uint32_t*>(dst + (int64_t)r * K) = c[r];
  }
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
  store_transposed(codes, c);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int f = 32 * j + (threadIdx.x >> 3), chunk = threadIdx.x & 7;
    const int k = kb * 128 + f, n = nb * 128 + 16 * chunk;
    if (k < K && n < N)
      *reinterpret_cast<uint4*>(q_t + (g * K + k) * N + n) = *transposed(codes, f, chunk);
  }
}

template <typename T>
void rows_launch(const void* x, int64_t x_rows, int64_t ld, const int32_t* row_idx, int64_t M,
                 int K, uint8_t* q, uint8_t* scale, cudaStream_t stream) {
  const int words = (int)(fp8_scale_pitch(K) / 4);
  const int64_t need = (M + 7) / 8;                        // CTAs with a row for every warp
  int64_t grid = (2 * RowsShape<T>::ctas * (int64_t)sm_count() + words - 1) / words;
  if (grid > need) grid = need;
  rows_kernel<T><<<dim3((unsigned)grid, (unsigned)words), 256, 0, stream>>>(
      static_cast<const T*>(x), x_rows, ld, row_idx, M, K, words, q,
      reinterpret_cast<uint32_t*>(scale));
}

template <typename T>
void cols_launch(const void* x, int64_t x_rows, int64_t ld, const int32_t* row_idx,
                 const int32_t* offsets, int G, int64_t M, int K, int64_t width, uint8_t* q_t,
                 uint8_t* scale_t, cudaStream_t stream) {
  const int words = (int)(fp8_scale_pitch(width) / 4);
  using S = ColsShape<T>;
  const int64_t units = (int64_t)((K + S::features - 1) / S::features) * (width / 128);
  const int64_t most = S::ctas * (int64_t)sm_count();  // CTAs at a time
  const int64_t run = (units + most - 1) / most;
  cols_kernel<T><<<(unsigned)((units + run - 1) / run), S::warps * 32, 0, stream>>>(
      static_cast<const T*>(x), x_rows, ld, row_idx, offsets, G, M, K, width, words, run, q_t,
      scale_t);
}

}  // namespace

int launch_fp8_rows(const void* x, int dtype, int64_t x_rows, int64_t ld, const int32_t* row_idx,
                    int64_t M, int K, uint8_t* q, uint8_t* scale, cudaStream_t stream) {
  if (dtype == QB_F32)
    rows_launch<float>(x, x_rows, ld, row_idx, M, K, q, scale, stream);
  else
    rows_launch<__nv_bfloat16>(x, x_rows, ld, row_idx, M, K, q, scale, stream);
  return launch_status();
}

int launch_fp8_cols(const void* x, int dtype, int64_t x_rows, int64_t ld, const int32_t* row_idx,
                    const int32_t* offsets, int G, int64_t M, int K, int64_t width, uint8_t* q_t,
                    uint8_t* scale_t, cudaStream_t stream) {
  if (dtype == QB_F32)
    cols_launch<float>(x, x_rows, ld, row_idx, offsets, G, M, K, width, q_t, scale_t, stream);
  else
    cols_launch<__nv_bfloat16>(x, x_rows, ld, row_idx, offsets, G, M, K, width, q_t, scale_t,
                               stream);
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
