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
// Both passes are bound by HBM: one read of the logits (and one write of the
// gradient).  A row is held by 8, 16 or 32 lanes, 4 consecutive columns of a
// lane to a load, so that the row's sums take 3 to 5 shuffles for up to 32
// values of a lane; each lane keeps its columns' P_e in registers over the
// CTA's rows.  The CTAs' sums are added in a fixed order by the last CTA of
// the batch to finish, so equal inputs give equal results.
#include <cuda_bf16.h>

#include "qb_device.cuh"
#include "qb_internal.h"

namespace qb {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kEps = 1e-20f;
// Tickets at the head of the workspace, the same number for every size, so
// that a workspace serves calls of several sizes in turn.  More than one CTA
// to a batch means fewer batches than kLossWaves * SMs.
constexpr int kTickets = 1024;
constexpr float kLog2e = 0x1.715476p+0f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

__device__ __forceinline__ void load_cols(const float* p, float (&x)[4]) {
  const float4 f = __ldg(reinterpret_cast<const float4*>(p));
  x[0] = f.x;
  x[1] = f.y;
  x[2] = f.z;
  x[3] = f.w;
}
__device__ __forceinline__ void load_cols(const __nv_bfloat16* p, float (&x)[4]) {
  const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
  x[0] = __uint_as_float(u.x << 16);
  x[1] = __uint_as_float(u.x & 0xFFFF0000u);
  x[2] = __uint_as_float(u.y << 16);
  x[3] = __uint_as_float(u.y & 0xFFFF0000u);
}

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

// Scores of a lane's J groups of four columns.  Sigmoid: s, and g = s (1 - s)
// where kGrad.  Softmax: s = exp(x - row max).  Inputs below -80 count as -80
// (s = 2e-35 there, far below the 1e-20 beside the sum); NaN stays NaN.
template <int SCORE, int J, int LPR, bool kGrad>
__device__ __forceinline__ void scores(float (&x)[J][4], const bool (&in)[J], float (&g)[J][4]) {
  if (SCORE == QB_SCORE_SIGMOID) {
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float e = ex2(__fmul_rn(max_nan(x[j][c], -80.0f), -kLog2e));
        const float s = in[j] ? rcp_approx(__fadd_rn(1.0f, e)) : 0.0f;
        x[j][c] = s;
        if (kGrad) g[j][c] = __fmul_rn(__fmul_rn(s, s), e);
      }
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) m = in[j] ? max_nan(m, x[j][c]) : m;
    m = row_max<LPR>(m);
    m = m == -INFINITY ? 0.0f : m;  // a row without any finite logit: all shares 0
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        x[j][c] = in[j] ? ex2(__fmul_rn(__fsub_rn(x[j][c], m), kLog2e)) : 0.0f;
  }
}

template <int SCORE, int J, int LPR>
__device__ __forceinline__ float row_total(const float (&s)[J][4]) {
  float t = 0.0f;
#pragma unroll
  for (int j = 0; j < J; ++j)
    t += __fadd_rn(__fadd_rn(s[j][0], s[j][1]), __fadd_rn(s[j][2], s[j][3]));
  return row_sum<LPR>(t);
}
template <int SCORE>
__device__ __forceinline__ float inverse_total(float t) {
  if (SCORE == QB_SCORE_SIGMOID) return __fdiv_rn(1.0f, __fadd_rn(t, kEps));
  return t == 0.0f ? 0.0f : __fdiv_rn(1.0f, t);
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
  unsigned* ticket;   // [batches], zero between calls
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
    const double nn = n > 0 ? (double)n : 1.0;
    a.loss[b] = (float)((double)t * a.coeff * a.E / (a.k * nn * nn));
    a.tokens[b] = n;
  }
}

template <typename T, int SCORE, int J, int LPR>
__global__ void __launch_bounds__(kThreads)
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
  const int64_t b = blockIdx.x / a.runs;
  const int64_t first = b * a.batch;
  const int64_t end_b = first + a.batch < a.N ? first + a.batch : a.N;
  int64_t lo = first + (blockIdx.x - b * a.runs) * a.run;
  if (lo > end_b) lo = end_b;
  const int64_t hi = lo + a.run < end_b ? lo + a.run : end_b;
  for (int e = threadIdx.x; e < a.E; e += kThreads) cnt[e] = 0;
  if (threadIdx.x == 0) live_tokens = 0;
  __syncthreads();

  // counts of the CTA's tokens
  const int64_t entries = (hi - lo) * a.k;
  for (int64_t i = threadIdx.x; i < entries; i += kThreads) {
    const int e = a.topk[lo * a.k + i];
    const bool live = !a.mask || a.mask[lo + i / a.k];
    if (live && (unsigned)e < (unsigned)a.E) atomicAdd(cnt + e, 1);
  }

  float acc[J][4];
  bool in[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    in[j] = (sub + LPR * j) * 4 < a.E;
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[j][c] = 0.0f;
  }
  int n = 0;
  for (int64_t r0 = lo + warp * kRows; r0 < hi; r0 += kWarps * kRows) {
    const int64_t r = r0 + lane / LPR;
    const bool live = r < hi && (!a.mask || a.mask[r]);
    float x[J][4], g[J][4];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      x[j][0] = x[j][1] = x[j][2] = x[j][3] = 0.0f;
      if (live && in[j]) load_cols(logits + r * a.E + (sub + LPR * j) * 4, x[j]);
    }
    scores<SCORE, J, LPR, false>(x, in, g);
    float inv = inverse_total<SCORE>(row_total<SCORE, J, LPR>(x));
    inv = live ? inv : 0.0f;
    n += live && sub == 0;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[j][c] = __fmaf_rn(x[j][c], inv, acc[j][c]);
  }
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
#pragma unroll
      for (int d = LPR; d < 32; d <<= 1) acc[j][c] += __shfl_xor_sync(0xffffffffu, acc[j][c], d);
      if (lane < LPR && in[j]) sum[warp * a.E + (sub + LPR * j) * 4 + c] = acc[j][c];
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
  if (a.runs == 1) {
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
      a.counts[b * a.E + e] = cnt[e];
      a.prob_sum[b * a.E + e] = sum[e];
    }
    write_loss(a, b, sum, cnt, live_tokens, red);
    return;
  }
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    a.part_sum[(int64_t)blockIdx.x * a.E + e] = sum[e];
    a.part_cnt[(int64_t)blockIdx.x * a.E + e] = cnt[e];
  }
  if (threadIdx.x == 0) a.part_tok[blockIdx.x] = live_tokens;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(a.ticket + b, 1u) == (unsigned)a.runs - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    float t = 0.0f;
    int c = 0;
#pragma unroll 8
    for (int i = 0; i < a.runs; ++i) {
      t += __ldcg(a.part_sum + (b * a.runs + i) * a.E + e);
      c += __ldcg(a.part_cnt + (b * a.runs + i) * a.E + e);
    }
    sum[e] = t;
    cnt[e] = c;
    a.counts[b * a.E + e] = c;
    a.prob_sum[b * a.E + e] = t;
  }
  if (threadIdx.x == 0) {
    live_tokens = 0;
    a.ticket[b] = 0;
  }
  __syncthreads();
  int m = 0;
  for (int i = threadIdx.x; i < a.runs; i += kThreads) m += __ldcg(a.part_tok + b * a.runs + i);
  if (m) atomicAdd(&live_tokens, m);
  __syncthreads();
  write_loss(a, b, sum, cnt, live_tokens, red);
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
__global__ void __launch_bounds__(kThreads)
    balance_grad_kernel(const T* __restrict__ logits, const GradArgs a) {
  constexpr int kRows = 32 / LPR;
  __shared__ long long total;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % LPR;
  const int64_t b = blockIdx.x / a.runs;
  const int64_t first = b * a.batch;
  const int64_t end_b = first + a.batch < a.N ? first + a.batch : a.N;
  int64_t lo = first + (blockIdx.x - b * a.runs) * a.run;
  if (lo > end_b) lo = end_b;
  const int64_t hi = lo + a.run < end_b ? lo + a.run : end_b;

  if (threadIdx.x == 0) total = 0;
  __syncthreads();
  long long mine = 0;
  for (int e = threadIdx.x; e < a.E; e += kThreads) mine += a.counts[b * a.E + e];
  if (mine) atomicAdd(reinterpret_cast<unsigned long long*>(&total), (unsigned long long)mine);
  __syncthreads();
  const int c0 = (int)(total / a.E);
  const int n = a.tokens[b];
  const double nn = n > 0 ? (double)n : 1.0;
  const float f = (float)((double)a.loss_grad[b] * a.coeff * a.E / (a.k * nn * nn));
  float w[J][4];
  bool in[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    in[j] = (sub + LPR * j) * 4 < a.E;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      w[j][c] = in[j] ? (float)(a.counts[b * a.E + (sub + LPR * j) * 4 + c] - c0) : 0.0f;
  }
  for (int64_t r0 = lo + warp * kRows; r0 < hi; r0 += kWarps * kRows) {
    const int64_t r = r0 + lane / LPR;
    const bool valid = r < hi;
    const bool live = valid && (!a.mask || a.mask[r]);
    float x[J][4], g[J][4];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      x[j][0] = x[j][1] = x[j][2] = x[j][3] = 0.0f;
      if (live && in[j]) load_cols(logits + r * a.E + (sub + LPR * j) * 4, x[j]);
    }
    scores<SCORE, J, LPR, true>(x, in, g);
    const float inv = inverse_total<SCORE>(row_total<SCORE, J, LPR>(x));
    float d = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) d = __fmaf_rn(w[j][c], x[j][c], d);
    d = __fmul_rn(row_sum<LPR>(d), inv);
    // the part of c0 that the 1e-20 beside the sum leaves
    if (SCORE == QB_SCORE_SIGMOID) d = __fmaf_rn(-(float)c0, __fmul_rn(kEps, inv), d);
    const float scale = __fmul_rn(f, inv);
    if (valid) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (!in[j]) continue;
        float o[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float s = SCORE == QB_SCORE_SIGMOID ? g[j][c] : x[j][c];
          o[c] = live ? __fmul_rn(__fmul_rn(s, scale), __fsub_rn(w[j][c], d)) : 0.0f;
        }
        float4* dst = reinterpret_cast<float4*>(a.grad + r * a.E + (sub + LPR * j) * 4);
        if (a.accumulate) {
          if (live) {
            const float4 old = *dst;
            *dst = make_float4(old.x + o[0], old.y + o[1], old.z + o[2], old.w + o[3]);
          }
        } else {
          *dst = make_float4(o[0], o[1], o[2], o[3]);
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
constexpr int kGradWaves = 8;

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
#define QB_BY_WIDTH(fn, T, S)                                          \
  (a.E <= 32    ? fn<T, S, 1, 8>(logits, a, ctas, stream)              \
   : a.E <= 64  ? fn<T, S, 2, 8>(logits, a, ctas, stream)              \
   : a.E <= 128 ? fn<T, S, 4, 8>(logits, a, ctas, stream)              \
   : a.E <= 256 ? fn<T, S, 8, 8>(logits, a, ctas, stream)              \
   : a.E <= 512 ? fn<T, S, 8, 16>(logits, a, ctas, stream)             \
                : fn<T, S, 8, 32>(logits, a, ctas, stream))
#define QB_BY_TYPE(fn)                                                                     \
  (dtype == QB_F32 ? (score == QB_SCORE_SIGMOID ? QB_BY_WIDTH(fn, float, QB_SCORE_SIGMOID) \
                                                : QB_BY_WIDTH(fn, float, QB_SCORE_SOFTMAX)) \
                   : (score == QB_SCORE_SIGMOID                                            \
                          ? QB_BY_WIDTH(fn, __nv_bfloat16, QB_SCORE_SIGMOID)               \
                          : QB_BY_WIDTH(fn, __nv_bfloat16, QB_SCORE_SOFTMAX)))

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
    if (batches > kTickets) return QB_EUNSUPPORTED;
    a.ticket = static_cast<unsigned*>(workspace);
    a.part_tok = reinterpret_cast<int*>(a.ticket + kTickets);
    a.part_cnt = a.part_tok + ctas;
    a.part_sum = reinterpret_cast<float*>(a.part_cnt + ctas * E);
  }
  return QB_BY_TYPE(launch_loss);
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
  return QB_BY_TYPE(launch_grad);
}

}  // namespace qb
