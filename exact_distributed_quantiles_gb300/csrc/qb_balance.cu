// qb_balance.cu -- the load-balance loss of a router with its per-expert
// counts, and the loss's gradient.
//
// The N tokens are split into consecutive local batches.  Of a batch's n live
// tokens, c_e top-k entries name expert e and p[i,e] is token i's share of
// expert e,
//   sigmoid  p = s / (sum_j s_j + 1e-20), s = 1 / (1 + exp(-x))
//   softmax  p = exp(x - max x) / sum_j exp(x_j - max x)
//   L = coeff * E / (k n^2) * sum_e c_e P_e,      P_e = sum_i p[i,e]
// The counts do not depend on x differentiably, so with
// w_e = dL * coeff * E / (k n^2) * c_e
//   sigmoid  dx_e = s_e (1 - s_e) / S * (w_e - sum_j w_j p_j)
//   softmax  dx_e = p_e * (w_e - sum_j w_j p_j)
// The difference is formed with c_e - c0 (c0 the counts' mean, a whole
// number) in place of c_e: shares sum to one, so c0 drops out exactly and the
// rounding of p no longer meets the counts' common part.
//
// Both passes are one read of the logits (and one write of the gradient).  A
// row is held by 8, 16 or 32 lanes, 4 consecutive columns of a lane to a load,
// so that the row's sums take 3 to 5 shuffles for up to 32 values of a lane;
// values are worked on in pairs (f32x2), the next row is read while the current
// one is worked on, and each lane keeps its columns' P_e in registers over the
// CTA's rows.  The CTAs' sums are added in a fixed order, sixteen by the last
// CTA of the sixteen to finish, so equal inputs give equal results.
// Measured: loss of 524288 x 256 fp32 logits 93 us (5.9 TB/s, HBM bound); of
// 262144 x 256 bf16 44 us (3.2 TB/s: two special-function operations a value,
// four warps a scheduler), its gradient 75 us (5.4 TB/s).
#include <cuda_bf16.h>

#include <cfloat>

#include "qb_device.cuh"
#include "qb_internal.h"

namespace qb {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kEps = 1e-20f;
// Tickets at the head of the workspace, the same number for every size, so
// that a workspace serves calls of several sizes in turn: one for each sixteen
// CTAs of a batch, and from the half on one for each batch.  More than one CTA
// to a batch means fewer batches than kLossWaves * SMs.
constexpr int kTickets = 2048;
constexpr float kLog2e = 0x1.715476p+0f;

// The .ftz form is the bare instruction; it flushes results below 2^-126, far
// under what 1 + e or a sum of scores keeps.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// rcp_approx for any input here: 1 / inf = 0 (a score of a very negative logit)
__device__ __forceinline__ f2_t rcp2(f2_t d) {
  float lo, hi;
  f2_unpack(d, lo, hi);
  return f2_pack(rcp_approx(lo), rcp_approx(hi));
}
__device__ __forceinline__ f2_t ex2_2(f2_t t) {
  float lo, hi;
  f2_unpack(t, lo, hi);
  return f2_pack(ex2(lo), ex2(hi));
}

// Four consecutive logits as they come from memory.  Columns behind the last
// expert count as -inf: their score is 0.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float4 f;
  __device__ __forceinline__ void load(const float* p) {
    f = __ldg(reinterpret_cast<const float4*>(p));
  }
  __device__ __forceinline__ void fill(float v) { f = make_float4(v, v, v, v); }
  __device__ __forceinline__ void values(float (&x)[4]) const {
    x[0] = f.x;
    x[1] = f.y;
    x[2] = f.z;
    x[3] = f.w;
  }
};
template <>
struct Raw<__nv_bfloat16> {
  uint2 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    u = __ldg(reinterpret_cast<const uint2*>(p));
  }
  __device__ __forceinline__ void fill(float v) {
    const uint32_t b = __float_as_uint(v) >> 16;
    u.x = u.y = b | b << 16;
  }
  __device__ __forceinline__ void values(float (&x)[4]) const {
    x[0] = __uint_as_float(u.x << 16);
    x[1] = __uint_as_float(u.x & 0xFFFF0000u);
    x[2] = __uint_as_float(u.y << 16);
    x[3] = __uint_as_float(u.y & 0xFFFF0000u);
  }
};

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int d = 1; d < LPR; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
template <int LPR>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int d = 1; d < LPR; d <<= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}

// One row's groups of four columns of a lane.
template <typename T, int J, int LPR>
__device__ __forceinline__ void load_row(const T* logits, int64_t r, bool live, int E, int sub,
                                         Raw<T> (&raw)[J]) {
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int col = (sub + LPR * j) * 4;
    if (col >= E)
      raw[j].fill(-INFINITY);
    else if (live)
      raw[j].load(logits + r * E + col);
    else
      raw[j].fill(0.0f);
  }
}

// Scores of a lane's J groups of four columns, in pairs.  Sigmoid: s, and
// g = s (1 - s) = s (s e) with e = exp(-x) where kGrad.  s e = 1 - s lies in
// [0, 1] and g is near s where s is small, so nothing vanishes before s does,
// far below the 1e-20 beside the sum (s s, in place of it, is subnormal from
// x = -44 on, where a row of such scores still has an ordinary gradient).
// Where e overflows s is 0, and the largest number in e's place gives g = 0.
// Softmax: s = exp(x - row max).  NaN stays NaN.
template <typename T, int SCORE, int J, int LPR, bool kGrad>
__device__ __forceinline__ void scores(const Raw<T> (&raw)[J], f2_t (&s)[J][2],
                                       f2_t (&g)[J][2]) {
  if (SCORE == QB_SCORE_SIGMOID) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float x[4];
      raw[j].values(x);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f2_t e = ex2_2(f2_mul(f2_pack(x[2 * h], x[2 * h + 1]), f2_splat(-kLog2e)));
        s[j][h] = rcp2(f2_add(e, f2_splat(1.0f)));
        if (kGrad) {
          float lo, hi;
          f2_unpack(e, lo, hi);
          const f2_t held = f2_pack(min_nan(lo, FLT_MAX), min_nan(hi, FLT_MAX));
          g[j][h] = f2_mul(s[j][h], f2_mul(s[j][h], held));
        }
      }
    }
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float x[4];
      raw[j].values(x);
#pragma unroll
      for (int c = 0; c < 4; ++c) m = max_nan(m, x[c]);
    }
    m = row_max<LPR>(m);
    m = m == -INFINITY ? 0.0f : m;  // a row without any finite logit: all shares 0
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float x[4];
      raw[j].values(x);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        s[j][h] = ex2_2(f2_mul(f2_sub(f2_pack(x[2 * h], x[2 * h + 1]), f2_splat(m)),
                               f2_splat(kLog2e)));
    }
  }
}

template <int J, int LPR>
__device__ __forceinline__ float row_total(const f2_t (&s)[J][2]) {
  f2_t t = f2_add(s[0][0], s[0][1]);
#pragma unroll
  for (int j = 1; j < J; ++j) t = f2_add(t, f2_add(s[j][0], s[j][1]));
  float lo, hi;
  f2_unpack(t, lo, hi);
  return row_sum<LPR>(__fadd_rn(lo, hi));
}
template <int SCORE>
__device__ __forceinline__ float inverse_total(float t) {
  if (SCORE == QB_SCORE_SIGMOID) return __frcp_rn(__fadd_rn(t, kEps));
  return t == 0.0f ? 0.0f : __frcp_rn(t);
}

// coeff * E / (k n^2), the weight of a batch of n live tokens; fp32, four
// roundings (fp64 would cost a microsecond of latency here).
__device__ __forceinline__ float batch_weight(float coeff, int E, int k, int n) {
  const float m = n > 0 ? (float)n : 1.0f;
  return __fdiv_rn(__fdiv_rn(__fmul_rn(coeff, (float)E), __fmul_rn((float)k, m)), m);
}

// ------------------------------------------------------------------ loss
struct LossArgs {
  const int32_t* topk;
  const uint8_t* mask;
  int64_t N, batch;   // tokens; tokens of a local batch
  int64_t run;        // tokens of a CTA
  int E, k, runs;     // runs: CTAs of a batch
  float coeff;
  int32_t* counts;    // [batches, E]
  int32_t* tokens;    // [batches]
  float* prob_sum;    // [batches, E]
  float* loss;        // [batches]
  // where runs > 1: every CTA's sums, and one ticket per batch
  float* part_sum;    // [batches * runs, E]
  int* part_cnt;      // [batches * runs, E]
  int* part_tok;      // [batches * runs]
  unsigned* ticket;   // [kTickets], zero between calls
};

// L of one batch from its sums in shared memory; every thread of the CTA.
__device__ __forceinline__ void write_loss(const LossArgs& a, int64_t b, const float* sum,
                                           const int* cnt, int n, float* red) {
  float v = 0.0f;
  for (int e = threadIdx.x; e < a.E; e += kThreads) v += __fmul_rn((float)cnt[e], sum[e]);
  v = row_sum<32>(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    float t = 0.0f;
    for (int w = 0; w < kWarps; ++w) t += red[w];
    a.loss[b] = __fmul_rn(t, batch_weight(a.coeff, a.E, a.k, n));
    a.tokens[b] = n;
  }
}

constexpr int kJoin = 16;  // CTAs whose sums one of them adds

// Adds n rows of sums and counts, `stride` rows apart, in their order.
__device__ __forceinline__ int join(const LossArgs& a, int64_t row, int n, int stride, float* sum,
                                    int* cnt) {
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    float t = 0.0f;
    int c = 0;
    for (int i0 = 0; i0 < n; i0 += 8) {
      float f[8];
      int k[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t at = (row + (int64_t)(i0 + i) * stride) * a.E + e;
        f[i] = i0 + i < n ? __ldcg(a.part_sum + at) : 0.0f;
        k[i] = i0 + i < n ? __ldcg(a.part_cnt + at) : 0;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        t += f[i];
        c += k[i];
      }
    }
    sum[e] = t;
    cnt[e] = c;
  }
  int m = 0;
  for (int i = 0; i < n; ++i) m += __ldcg(a.part_tok + row + (int64_t)i * stride);
  return m;
}

// Whether this CTA is the last of n to come here; the ticket is left at zero.
__device__ __forceinline__ bool last_of(unsigned* ticket, unsigned n, bool* flag) {
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    *flag = atomicAdd(ticket, 1u) == n - 1;
    if (*flag) *ticket = 0;
  }
  __syncthreads();
  const bool last = *flag;
  if (last) __threadfence();
  return last;
}

__device__ __forceinline__ void write_part(const LossArgs& a, int64_t row, const float* sum,
                                           const int* cnt, int tokens) {
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    a.part_sum[row * a.E + e] = sum[e];
    a.part_cnt[row * a.E + e] = cnt[e];
  }
  if (threadIdx.x == 0) a.part_tok[row] = tokens;
}

template <typename T, int SCORE, int J, int LPR>
__global__ void __launch_bounds__(kThreads, 2)
    balance_loss_kernel(const T* __restrict__ logits, const LossArgs a) {
  constexpr int kRows = 32 / LPR;  // rows of a warp at a time
  extern __shared__ float sm[];
  float* sum = sm;                                       // [kWarps][E], then [E]
  int* cnt = reinterpret_cast<int*>(sm + kWarps * a.E);  // [E]
  __shared__ int live_tokens;
  __shared__ bool last;
  __shared__ float red[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % LPR;
  const int64_t b = blockIdx.x / (unsigned)a.runs;
  const int run_no = (int)(blockIdx.x % (unsigned)a.runs);
  const int64_t first = b * a.batch;
  const int64_t end_b = first + a.batch < a.N ? first + a.batch : a.N;
  int64_t lo = first + run_no * a.run;
  if (lo > end_b) lo = end_b;
  const int64_t hi = lo + a.run < end_b ? lo + a.run : end_b;
  for (int e = threadIdx.x; e < a.E; e += kThreads) cnt[e] = 0;
  if (threadIdx.x == 0) live_tokens = 0;
  __syncthreads();

  f2_t acc[J][2];
#pragma unroll
  for (int j = 0; j < J; ++j) acc[j][0] = acc[j][1] = 0;
  int n = 0;
  // the warp's rows of a step have kRows * k (at most 60) entries: one or two a lane
  const int entries = kRows * a.k, row_a = lane / a.k, row_b = (lane + 32) / a.k;
  int64_t r0 = lo + warp * kRows;
  const auto read = [&](int64_t r0, Raw<T>(&raw)[J], bool& live, int& ea, int& eb) {
    const int64_t r = r0 + lane / LPR;
    live = r < hi && (!a.mask || a.mask[r]);
    ea = eb = -1;
    if (lane < entries && r0 + row_a < hi) ea = __ldg(a.topk + r0 * a.k + lane);
    if (lane + 32 < entries && r0 + row_b < hi) eb = __ldg(a.topk + r0 * a.k + lane + 32);
    load_row<T, J, LPR>(logits, r, live, a.E, sub, raw);
  };
  Raw<T> raw[J];
  bool live = false;
  int ea = -1, eb = -1;
  if (r0 < hi) read(r0, raw, live, ea, eb);
  while (r0 < hi) {
    f2_t s[J][2], g[J][2];
    scores<T, SCORE, J, LPR, false>(raw, s, g);
    const bool now = live;
    const int ca = ea, cb = eb;
    r0 += kWarps * kRows;
    if (r0 < hi) read(r0, raw, live, ea, eb);
    float inv = inverse_total<SCORE>(row_total<J, LPR>(s));
    inv = now ? inv : 0.0f;
    n += now && sub == 0;
    const unsigned rows = __ballot_sync(0xffffffffu, now);  // bit LPR * i: row i is live
    if ((unsigned)ca < (unsigned)a.E && (rows >> (row_a * LPR) & 1u)) atomicAdd(cnt + ca, 1);
    if ((unsigned)cb < (unsigned)a.E && (rows >> (row_b * LPR) & 1u)) atomicAdd(cnt + cb, 1);
    const f2_t inv2 = f2_splat(inv);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      acc[j][0] = f2_fma(s[j][0], inv2, acc[j][0]);
      acc[j][1] = f2_fma(s[j][1], inv2, acc[j][1]);
    }
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    float v[4];
    f2_unpack(acc[j][0], v[0], v[1]);
    f2_unpack(acc[j][1], v[2], v[3]);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
#pragma unroll
      for (int d = LPR; d < 32; d <<= 1) v[c] += __shfl_xor_sync(0xffffffffu, v[c], d);
    }
    const int col = (sub + LPR * j) * 4;
    if (lane < LPR && col < a.E)
      *reinterpret_cast<float4*>(sum + warp * a.E + col) = make_float4(v[0], v[1], v[2], v[3]);
  }
  if (n) atomicAdd(&live_tokens, n);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t += sum[w * a.E + e];
    sum[e] = t;  // this thread alone reads column e of the warps' rows
  }
  __syncthreads();
  int tokens = live_tokens;
  if (a.runs > 1) {
    // sixteen CTAs' sums by the last of them, then those by the last of these
    const int64_t row = b * a.runs;
    const int group = run_no / kJoin, groups = (a.runs + kJoin - 1) / kJoin;
    const int here = a.runs - group * kJoin < kJoin ? a.runs - group * kJoin : kJoin;
    write_part(a, row + run_no, sum, cnt, tokens);
    if (!last_of(a.ticket + b * groups + group, here, &last)) return;
    tokens = join(a, row + group * kJoin, here, 1, sum, cnt);
    __syncthreads();
    if (groups > 1) {
      write_part(a, row + group * kJoin, sum, cnt, tokens);
      if (!last_of(a.ticket + kTickets / 2 + b, groups, &last)) return;
      tokens = join(a, row, groups, kJoin, sum, cnt);
      __syncthreads();
    }
  }
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    a.counts[b * a.E + e] = cnt[e];
    a.prob_sum[b * a.E + e] = sum[e];
  }
  write_loss(a, b, sum, cnt, tokens, red);
}

// ------------------------------------------------------------------ gradient
struct GradArgs {
  const uint8_t* mask;
  const int32_t* counts;
  const int32_t* tokens;
  const float* loss_grad;
  int64_t N, batch, run;
  int E, k, runs, accumulate;
  float coeff;
  float* grad;
};

template <typename T, int SCORE, int J, int LPR>
__global__ void __launch_bounds__(kThreads, J > 4 ? 2 : 3)
    balance_grad_kernel(const T* __restrict__ logits, const GradArgs a) {
  constexpr int kRows = 32 / LPR;
  __shared__ long long total;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % LPR;
  const int64_t b = blockIdx.x / (unsigned)a.runs;
  const int64_t first = b * a.batch;
  const int64_t end_b = first + a.batch < a.N ? first + a.batch : a.N;
  int64_t lo = first + (int64_t)(blockIdx.x % (unsigned)a.runs) * a.run;
  if (lo > end_b) lo = end_b;
  const int64_t hi = lo + a.run < end_b ? lo + a.run : end_b;

  const auto read = [&](int64_t r0, Raw<T>(&raw)[J], bool& live) {
    const int64_t r = r0 + lane / LPR;
    live = r < hi && (!a.mask || a.mask[r]);
    load_row<T, J, LPR>(logits, r, live, a.E, sub, raw);
  };
  int64_t r0 = lo + warp * kRows;
  Raw<T> raw[J];
  bool live = false;
  if (r0 < hi) read(r0, raw, live);  // on its way while the counts are read

  const int n = a.tokens[b];
  const float loss_grad = a.loss_grad[b];
  if (threadIdx.x == 0) total = 0;
  __syncthreads();
  long long mine = 0;
  for (int e = threadIdx.x; e < a.E; e += kThreads) mine += a.counts[b * a.E + e];
  if (mine) atomicAdd(reinterpret_cast<unsigned long long*>(&total), (unsigned long long)mine);
  __syncthreads();
  const int c0 = (int)__fdiv_rn((float)total, (float)a.E);  // any number near the mean serves
  const float f = __fmul_rn(loss_grad, batch_weight(a.coeff, a.E, a.k, n));
  f2_t w[J][2];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int col = (sub + LPR * j) * 4;
    float v[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = col < a.E ? (float)(a.counts[b * a.E + col + c] - c0) : 0.0f;
    w[j][0] = f2_pack(v[0], v[1]);
    w[j][1] = f2_pack(v[2], v[3]);
  }
  while (r0 < hi) {
    f2_t s[J][2], g[J][2];
    scores<T, SCORE, J, LPR, true>(raw, s, g);
    const int64_t r = r0 + lane / LPR;
    const bool now = live;
    r0 += kWarps * kRows;
    if (r0 < hi) read(r0, raw, live);
    const float inv = inverse_total<SCORE>(row_total<J, LPR>(s));
    f2_t d2 = f2_mul(w[0][0], s[0][0]);
    d2 = f2_fma(w[0][1], s[0][1], d2);
#pragma unroll
    for (int j = 1; j < J; ++j) {
      d2 = f2_fma(w[j][0], s[j][0], d2);
      d2 = f2_fma(w[j][1], s[j][1], d2);
    }
    float d, dh;
    f2_unpack(d2, d, dh);
    d = __fmul_rn(row_sum<LPR>(__fadd_rn(d, dh)), inv);
    // the part of c0 that the 1e-20 beside the sum leaves
    if (SCORE == QB_SCORE_SIGMOID) d = __fmaf_rn(-(float)c0, __fmul_rn(kEps, inv), d);
    const f2_t front = f2_splat(__fmul_rn(f, inv)), mid = f2_splat(d);
    if (r < hi) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int col = (sub + LPR * j) * 4;
        if (col >= a.E) continue;
        float o[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f2_t v = SCORE == QB_SCORE_SIGMOID ? g[j][h] : s[j][h];
          f2_unpack(f2_mul(f2_mul(v, front), f2_sub(w[j][h], mid)), o[2 * h], o[2 * h + 1]);
        }
        float4* dst = reinterpret_cast<float4*>(a.grad + r * a.E + col);
        if (a.accumulate) {
          if (now) {
            const float4 old = *dst;
            *dst = make_float4(old.x + o[0], old.y + o[1], old.z + o[2], old.w + o[3]);
          }
        } else {
          *dst = now ? make_float4(o[0], o[1], o[2], o[3]) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
      }
    }
  }
}

// CTAs of a batch: enough in all to fill the GPU `waves` times over, and no
// fewer than 64 tokens for each.
void split(int64_t N, int64_t batch, int waves, int64_t& batches, int64_t& runs, int64_t& run) {
  batches = (N + batch - 1) / batch;
  runs = (waves * (int64_t)sm_count() + batches - 1) / batches;
  const int64_t most = (batch + 63) / 64;
  if (runs > most) runs = most;
  run = ((batch + runs - 1) / runs + 31) / 32 * 32;
  runs = (batch + run - 1) / run;
}

constexpr int kLossWaves = 2;
constexpr int kGradWaves = 3;

template <typename T, int SCORE, int J, int LPR>
int launch_loss(const void* logits, const LossArgs& a, int64_t ctas, cudaStream_t stream) {
  const int smem = (kWarps + 1) * a.E * 4;
  balance_loss_kernel<T, SCORE, J, LPR>
      <<<(unsigned)ctas, kThreads, smem, stream>>>(static_cast<const T*>(logits), a);
  return launch_status();
}
template <typename T, int SCORE, int J, int LPR>
int launch_grad(const void* logits, const GradArgs& a, int64_t ctas, cudaStream_t stream) {
  balance_grad_kernel<T, SCORE, J, LPR>
      <<<(unsigned)ctas, kThreads, 0, stream>>>(static_cast<const T*>(logits), a);
  return launch_status();
}

// Lanes of a row and groups of four columns of a lane, by the expert count.
// The loss keeps up to 32 columns of a lane; the gradient, which holds a row's
// scores, their derivatives, the counts and the next row, 16 where it can.
#define QB_LOSS_BY_WIDTH(T, S)                                              \
  (a.E <= 32    ? launch_loss<T, S, 1, 8>(logits, a, ctas, stream)          \
   : a.E <= 64  ? launch_loss<T, S, 2, 8>(logits, a, ctas, stream)          \
   : a.E <= 128 ? launch_loss<T, S, 4, 8>(logits, a, ctas, stream)          \
   : a.E <= 192 ? launch_loss<T, S, 6, 8>(logits, a, ctas, stream)          \
   : a.E <= 256 ? launch_loss<T, S, 8, 8>(logits, a, ctas, stream)          \
   : a.E <= 384 ? launch_loss<T, S, 6, 16>(logits, a, ctas, stream)         \
   : a.E <= 512 ? launch_loss<T, S, 8, 16>(logits, a, ctas, stream)         \
                : launch_loss<T, S, 8, 32>(logits, a, ctas, stream))
#define QB_GRAD_BY_WIDTH(T, S)                                              \
  (a.E <= 32    ? launch_grad<T, S, 1, 8>(logits, a, ctas, stream)          \
   : a.E <= 64  ? launch_grad<T, S, 2, 8>(logits, a, ctas, stream)          \
   : a.E <= 128 ? launch_grad<T, S, 4, 8>(logits, a, ctas, stream)          \
   : a.E <= 192 ? launch_grad<T, S, 3, 16>(logits, a, ctas, stream)         \
   : a.E <= 256 ? launch_grad<T, S, 4, 16>(logits, a, ctas, stream)         \
   : a.E <= 384 ? launch_grad<T, S, 3, 32>(logits, a, ctas, stream)         \
   : a.E <= 512 ? launch_grad<T, S, 4, 32>(logits, a, ctas, stream)         \
                : launch_grad<T, S, 8, 32>(logits, a, ctas, stream))
#define QB_BY_TYPE(by_width)                                                      \
  (dtype == QB_F32                                                                \
       ? (score == QB_SCORE_SIGMOID ? by_width(float, QB_SCORE_SIGMOID)           \
                                    : by_width(float, QB_SCORE_SOFTMAX))          \
       : (score == QB_SCORE_SIGMOID ? by_width(__nv_bfloat16, QB_SCORE_SIGMOID)   \
                                    : by_width(__nv_bfloat16, QB_SCORE_SOFTMAX)))

}  // namespace

int64_t balance_workspace_bytes(int64_t N, int E, int64_t batch) {
  int64_t batches, runs, run;
  split(N, batch, kLossWaves, batches, runs, run);
  if (runs == 1) return 0;
  return kTickets * 4 + batches * runs * ((int64_t)E * 8 + 4);
}

int launch_balance_loss(const void* logits, int dtype, const int32_t* topk, const uint8_t* mask,
                        int64_t N, int E, int k, int64_t batch, int score, float coeff,
                        int32_t* counts, int32_t* tokens, float* prob_sum, float* loss,
                        void* workspace, cudaStream_t stream) {
  int64_t batches, runs, run;
  split(N, batch, kLossWaves, batches, runs, run);
  const int64_t ctas = batches * runs;
  LossArgs a{topk, mask, N, batch, run, E, k, (int)runs, coeff, counts, tokens, prob_sum, loss,
             nullptr, nullptr, nullptr, nullptr};
  if (runs > 1) {
    if (batches * ((runs + kJoin - 1) / kJoin) > kTickets / 2) return QB_EUNSUPPORTED;
    a.ticket = static_cast<unsigned*>(workspace);
    a.part_tok = reinterpret_cast<int*>(a.ticket + kTickets);
    a.part_cnt = a.part_tok + ctas;
    a.part_sum = reinterpret_cast<float*>(a.part_cnt + ctas * E);
  }
  return QB_BY_TYPE(QB_LOSS_BY_WIDTH);
}

int launch_balance_grad(const void* logits, int dtype, const uint8_t* mask, const int32_t* counts,
                        const int32_t* tokens, const float* loss_grad, int64_t N, int E, int k,
                        int64_t batch, int score, float coeff, float* grad, int accumulate,
                        cudaStream_t stream) {
  int64_t batches, runs, run;
  split(N, batch, kGradWaves, batches, runs, run);
  const int64_t ctas = batches * runs;
  const GradArgs a{mask, counts, tokens, loss_grad, N, batch, run, E, k, (int)runs, accumulate,
                   coeff, grad};
  return QB_BY_TYPE(QB_GRAD_BY_WIDTH);
}

}  // namespace qb
