// qb_api.cu -- the extern "C" entry points of libqb: argument validation on
// the host, then one or more kernel launches on the caller's stream.  No
// entry point allocates memory or synchronises (except qb_device_status).
#include <mutex>

#include "qb_internal.h"

namespace qb {
namespace {

constexpr int kMaxDevices = 64;

// The device status word, one per device that loads the module.
__device__ int g_status_word;

struct PerDevice {
  std::once_flag once;
  int* status = nullptr;
  int sms = 0;
  bool ok = false;
};
PerDevice g_dev[kMaxDevices];

PerDevice* current() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  PerDevice* d = &g_dev[dev];
  std::call_once(d->once, [d, dev] {
    void* p = nullptr;
    int sms = 0;
    if (cudaGetSymbolAddress(&p, g_status_word) != cudaSuccess) return;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return;
    d->status = static_cast<int*>(p);
    d->sms = sms;
    d->ok = true;
  });
  return d->ok ? d : nullptr;
}

}  // namespace

int* device_status_ptr() {
  PerDevice* d = current();
  return d ? d->status : nullptr;
}

int sm_count() {
  PerDevice* d = current();
  return d ? d->sms : 1;
}

}  // namespace qb

using namespace qb;

namespace {

int check_route_args(const void* logits, int dtype, const float* bias, int64_t N, int E, int k) {
  if (!logits || !bias) return QB_EINVAL;
  if (dtype != QB_F32 && dtype != QB_BF16) return QB_EINVAL;
  if (!aligned16(logits)) return QB_EINVAL;
  if (N < 0) return QB_EINVAL;
  if (N > INT32_MAX) return QB_EOVERFLOW;
  if (!supported_E(E)) return QB_EUNSUPPORTED;
  if (k < 1 || k >= E) return QB_EINVAL;
  if (k > 15) return QB_EUNSUPPORTED;
  return QB_OK;
}

int router_gemm_hist_hi(const void* hidden, const void* w_t, int64_t M, int H, int E, int k,
                        const float* bias, float* logits_out, int32_t* hist_hi,
                        uint16_t* keys_out, int32_t* topk_out, float* alpha_out, void* stream,
                        bool chained) {
  if (!hidden || !w_t || !bias || !hist_hi) return QB_EINVAL;
  if (!aligned16(hidden) || !aligned16(w_t)) return QB_EINVAL;
  if ((logits_out && !aligned16(logits_out)) || (keys_out && !aligned16(keys_out)))
    return QB_EINVAL;
  if (M < 0) return QB_EINVAL;
  if (M > INT32_MAX) return QB_EOVERFLOW;
  if (E < 32 || E > 256 || E % 32 != 0 || H < 64 || H % 64 != 0) return QB_EUNSUPPORTED;
  if (k < 1 || k >= E) return QB_EINVAL;
  if (k > 15) return QB_EUNSUPPORTED;
  if (E != 256 && !logits_out) return QB_EUNSUPPORTED;
  if (M == 0) return QB_OK;
  if (E == 256)
    return launch_router_gemm_route(hidden, w_t, M, H, k, bias, hist_hi, keys_out, topk_out,
                                    alpha_out, logits_out, as_stream(stream), chained);
  // Other expert counts: the plain GEMM into logits_out, then the routing
  // pass on those logits (two launches; the fused epilogue is built for 256
  // experts).  The results are the same: the fused kernel equals the routing
  // pass run on its own logits.
  int st = launch_router_gemm(hidden, w_t, M, H, E, logits_out, as_stream(stream));
  if (st != QB_OK) return st;
  return launch_route_hi(logits_out, QB_F32, bias, M, E, k, hist_hi, keys_out, topk_out,
                         alpha_out, nullptr, nullptr, 0, as_stream(stream));
}

int k3_route_hist_impl(const void* logits, int dtype, const float* bias, int64_t N, int E, int k,
                       const float* bounds, int nbins, int32_t* hist, float* alpha_out,
                       void* stream, bool chained) {
  int st = check_route_args(logits, dtype, bias, N, E, k);
  if (st != QB_OK) return st;
  if (!bounds || !hist || !alpha_out) return QB_EINVAL;
  if ((reinterpret_cast<uintptr_t>(alpha_out) & 3u) != 0) return QB_EINVAL;
  if (nbins < 1 || nbins > 65536) return QB_EINVAL;
  if (N == 0) return QB_OK;
  cudaStream_t s = as_stream(stream);
  if (E == 256)
    st = dtype == QB_F32 ? launch_route256_alpha_f32(logits, bias, N, k, alpha_out, s, chained)
                         : launch_route256_alpha_bf16(logits, bias, N, k, alpha_out, s, chained);
  else
    st = launch_route_k3(logits, dtype, bias, N, E, k, nullptr, nullptr, nullptr, alpha_out,
                         nullptr, bounds, nbins, s);
  if (st != QB_OK) return st;
  return launch_k3_count(logits, dtype, alpha_out, N, E, bounds, nbins, hist, s);
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool is_dtype(int d) { return d == QB_F32 || d == QB_BF16; }

int check_balance_args(const void* logits, int dtype, int64_t N, int E, int k,
                       int64_t batch_tokens, int score) {
  if ((N > 0 && !logits) || !aligned16(logits) || !is_dtype(dtype)) return QB_EINVAL;
  if (score != QB_SCORE_SIGMOID && score != QB_SCORE_SOFTMAX) return QB_EINVAL;
  if (N < 0 || batch_tokens < 0) return QB_EINVAL;
  if (N > INT32_MAX) return QB_EOVERFLOW;
  if (!supported_E(E)) return QB_EUNSUPPORTED;
  if (k < 1 || k >= E) return QB_EINVAL;
  if (k > 15) return QB_EUNSUPPORTED;
  return N * k > INT32_MAX ? QB_EOVERFLOW : QB_OK;
}

// Groups of M rows: their number and where their offsets are.
int check_groups(const int32_t* offsets, int G, int64_t M) {
  if (G < 1 || (!offsets && G != 1) || !aligned4(offsets)) return QB_EINVAL;
  if (G > kMaxGroups) return QB_EUNSUPPORTED;
  if (M < 0) return QB_EINVAL;
  return M > INT32_MAX - 127 * kMaxGroups ? QB_EOVERFLOW : QB_OK;
}

int check_source(const void* x, int dtype, int64_t x_rows, int64_t ld, const int32_t* row_idx,
                 int64_t M, int K) {
  // no rows, no address: an empty tensor has none
  if ((x_rows > 0 && !x) || !aligned16(x) || !is_dtype(dtype) || !aligned4(row_idx))
    return QB_EINVAL;
  if (K < 16 || K % 16 != 0 || ld < K || ld % 16 != 0 || x_rows < 0 || M < 0) return QB_EINVAL;
  if (!row_idx && x_rows < M) return QB_EINVAL;
  return M > INT32_MAX || x_rows > INT32_MAX ? QB_EOVERFLOW : QB_OK;
}

// The weight gradient of one group without tokens: zeros, or what was there.
int launch_no_wgrad(int N, int K, void* out, int out_dtype, int accumulate, cudaStream_t s) {
  if (accumulate) return QB_OK;
  const size_t bytes = (size_t)N * (size_t)K * (out_dtype == QB_F32 ? 4 : 2);
  if (cudaMemsetAsync(out, 0, bytes, s) == cudaSuccess) return QB_OK;
  (void)cudaGetLastError();
  return QB_ECUDA;
}
}  // namespace

extern "C" {

const char* qb_status_string(int status) {
  switch (status) {
    case QB_OK:
      return "ok";
    case QB_EINVAL:
      return "invalid argument (null or misaligned pointer, bad size or rank)";
    case QB_EUNSUPPORTED:
      return "unsupported E or k (E a multiple of 32 up to 1024, 1 <= k <= 15, k < E)";
    case QB_ECUDA:
      return "CUDA launch or runtime error";
    case QB_EOVERFLOW:
      return "count would overflow its int32 counter";
    case QB_EDEVICE:
      return "a kernel reported a device-side error (bounded wait timed out)";
    default:
      return "unknown status";
  }
}

const char* qb_version(void) { return "libqb 0.1 (sm_103a)"; }

int64_t qb_rank(int64_t n_pool, int E, int k) {
  if (n_pool < 1 || E < 1 || k < 1 || k >= E) return QB_EINVAL;
  if (n_pool > INT64_MAX / 64) return QB_EOVERFLOW;
  return ((int64_t)k * n_pool + E - 1) / E;
}

int qb_sigmoid(const float* x, float* s, int64_t n, void* stream) {
  if (n < 0 || (n > 0 && (!x || !s))) return QB_EINVAL;
  return launch_sigmoid(x, s, n, 0, as_stream(stream));
}

int qb_sigmoid_scalar(const float* x, float* s, int64_t n, void* stream) {
  if (n < 0 || (n > 0 && (!x || !s))) return QB_EINVAL;
  return launch_sigmoid(x, s, n, 1, as_stream(stream));
}

int qb_selftest_wait_timeout(int64_t polls, void* stream) {
  if (polls < 1 || polls > (int64_t)1 << 24) return QB_EINVAL;
  return launch_wait_timeout_selftest((uint32_t)polls, as_stream(stream));
}

int qb_zero_i32(int32_t* p, int64_t n, void* stream) {
  if (n < 0 || (n > 0 && !p)) return QB_EINVAL;
  return launch_zero_i32(p, n, as_stream(stream));
}

int qb_route_hist_hi(const void* logits, int dtype, const float* bias, int64_t N, int E, int k,
                     int32_t* hist_hi, uint16_t* keys_out, int32_t* topk_out, float* alpha_out,
                     void* stream) {
  int st = check_route_args(logits, dtype, bias, N, E, k);
  if (st != QB_OK) return st;
  if (!hist_hi) return QB_EINVAL;
  if (keys_out && !aligned16(keys_out)) return QB_EINVAL;
  if (N == 0) return QB_OK;
  return launch_route_hi(logits, dtype, bias, N, E, k, hist_hi, keys_out, topk_out, alpha_out,
                         nullptr, nullptr, 0, as_stream(stream));
}

int qb_route_hist_hi_next(const void* logits, int dtype, const float* bias, int64_t N, int E,
                          int k, int32_t* hist_hi, uint16_t* keys_out, int32_t* topk_out,
                          float* alpha_out, void* stream) {
  int st = check_route_args(logits, dtype, bias, N, E, k);
  if (st != QB_OK) return st;
  if (!hist_hi) return QB_EINVAL;
  if (keys_out && !aligned16(keys_out)) return QB_EINVAL;
  if (N == 0) return QB_OK;
  if (E == 256 && dtype == QB_F32)
    return launch_route256_hi_f32(logits, bias, N, k, hist_hi, keys_out, topk_out, alpha_out,
                                  as_stream(stream), true);
  if (E == 256)
    return launch_route256_hi_bf16(logits, bias, N, k, hist_hi, keys_out, topk_out, alpha_out,
                                   as_stream(stream), true);
  return launch_route_hi(logits, dtype, bias, N, E, k, hist_hi, keys_out, topk_out, alpha_out,
                         nullptr, nullptr, 0, as_stream(stream));
}

int qb_select_hi(const int32_t* hist_hi, int E, int64_t r, int32_t* sel, int32_t* r_lo,
                 void* stream) {
  if (!hist_hi || !sel || !r_lo) return QB_EINVAL;
  if (!supported_E(E)) return QB_EUNSUPPORTED;
  if (r < 1) return QB_EINVAL;
  if (r > INT32_MAX) return QB_EOVERFLOW;
  return launch_select_hi(hist_hi, E, r, sel, r_lo, as_stream(stream));
}

int qb_keys_hist_lo(const uint16_t* keys, int64_t N, int E, const int32_t* sel,
                    int32_t* hist_lo, void* stream) {
  if (!keys || !sel || !hist_lo) return QB_EINVAL;
  if (!aligned16(keys)) return QB_EINVAL;
  if (N < 0) return QB_EINVAL;
  if (N > INT32_MAX) return QB_EOVERFLOW;
  if (!supported_E(E)) return QB_EUNSUPPORTED;
  if (N == 0) return QB_OK;
  return launch_keys_hist_lo(keys, N, E, sel, hist_lo, as_stream(stream));
}

int qb_route_hist_lo(const void* logits, int dtype, const float* bias, int64_t N, int E, int k,
                     const int32_t* sel, int32_t* hist_lo, void* stream) {
  int st = check_route_args(logits, dtype, bias, N, E, k);
  if (st != QB_OK) return st;
  if (!sel || !hist_lo) return QB_EINVAL;
  if (N == 0) return QB_OK;
  return launch_route_lo(logits, dtype, bias, N, E, k, hist_lo, nullptr, nullptr, nullptr, sel,
                         nullptr, 0, as_stream(stream));
}

int qb_finalize(int32_t* hist_hi, int32_t* hist_lo, const int32_t* sel, const int32_t* r_lo,
                int E, float* bias_out, uint16_t* qkey_out, int reset, void* stream) {
  if (!hist_lo || !sel || !r_lo || !bias_out) return QB_EINVAL;
  if (reset && !hist_hi) return QB_EINVAL;
  if (!supported_E(E)) return QB_EUNSUPPORTED;
  return launch_finalize(hist_hi, hist_lo, sel, r_lo, E, bias_out, qkey_out, reset,
                         as_stream(stream));
}

int k3_route_hist(const void* logits, int dtype, const float* bias, int64_t N, int E, int k,
                  const float* bounds, int nbins, int32_t* hist, float* alpha_out,
                  void* stream) {
  return k3_route_hist_impl(logits, dtype, bias, N, E, k, bounds, nbins, hist, alpha_out, stream,
                            false);
}

int k3_route_hist_next(const void* logits, int dtype, const float* bias, int64_t N, int E,
                       int k, const float* bounds, int nbins, int32_t* hist, float* alpha_out,
                       void* stream) {
  return k3_route_hist_impl(logits, dtype, bias, N, E, k, bounds, nbins, hist, alpha_out, stream,
                            true);
}

int k3_finalize(int32_t* hist, int E, int nbins, int64_t r, float* bounds, float* bias_out,
                int reset, void* stream) {
  if (!hist || !bounds || !bias_out) return QB_EINVAL;
  if (!supported_E(E)) return QB_EUNSUPPORTED;
  if (nbins < 1 || nbins > 65536) return QB_EINVAL;
  if (r < 1) return QB_EINVAL;
  if (r > INT32_MAX) return QB_EOVERFLOW;
  return launch_k3_finalize(hist, E, nbins, r, bounds, bias_out, reset, as_stream(stream));
}

int lei_inject(float* grad, const int32_t* topk_idx, int64_t N, int E, int k, float eta,
               int64_t batch_tokens, float* workspace, void* stream) {
  if (!grad || !topk_idx || !workspace) return QB_EINVAL;
  if (!aligned16(grad) || !aligned16(workspace)) return QB_EINVAL;
  if (N < 0 || batch_tokens < 0) return QB_EINVAL;
  if (!supported_E(E)) return QB_EUNSUPPORTED;
  if (k < 1 || k >= E) return QB_EINVAL;
  if (N == 0) return QB_OK;
  if (batch_tokens == 0 || batch_tokens > N) batch_tokens = N;
  if (N > INT32_MAX) return QB_EOVERFLOW;
  const int64_t nb = (N + batch_tokens - 1) / batch_tokens;
  if (nb > INT32_MAX) return QB_EINVAL;
  return launch_lei(grad, topk_idx, N, E, k, eta, batch_tokens, workspace, as_stream(stream));
}

int lei_rho(const int32_t* topk_idx, int64_t N, int E, int k, float eta, int64_t batch_tokens,
            float* workspace, void* stream) {
  if (!topk_idx || !workspace) return QB_EINVAL;
  if (!aligned16(workspace)) return QB_EINVAL;
  if (N < 0 || batch_tokens < 0) return QB_EINVAL;
  if (!supported_E(E)) return QB_EUNSUPPORTED;
  if (k < 1 || k >= E) return QB_EINVAL;
  if (N == 0) return QB_OK;
  if (batch_tokens == 0 || batch_tokens > N) batch_tokens = N;
  if (N > INT32_MAX) return QB_EOVERFLOW;
  const int64_t nb = (N + batch_tokens - 1) / batch_tokens;
  if (nb > INT32_MAX) return QB_EINVAL;
  return launch_lei_rho(topk_idx, N, E, k, eta, batch_tokens, workspace, as_stream(stream));
}

int lei_apply(float* grad, int64_t N, int E, int64_t batch_tokens, const float* workspace,
              void* stream) {
  if (!grad || !workspace) return QB_EINVAL;
  if (!aligned16(grad) || !aligned16(workspace)) return QB_EINVAL;
  if (N < 0 || batch_tokens < 0) return QB_EINVAL;
  if (!supported_E(E)) return QB_EUNSUPPORTED;
  if (N == 0) return QB_OK;
  if (batch_tokens == 0 || batch_tokens > N) batch_tokens = N;
  if (N > INT32_MAX) return QB_EOVERFLOW;
  return launch_lei_apply(grad, N, E, batch_tokens, workspace, as_stream(stream));
}

int lei_apply_overlap(float* grad, int64_t N, int E, int64_t batch_tokens, const float* workspace,
                      void* stream) {
  if (!grad || !workspace) return QB_EINVAL;
  if (!aligned16(grad) || !aligned16(workspace)) return QB_EINVAL;
  if (N < 0 || batch_tokens < 0) return QB_EINVAL;
  if (!supported_E(E)) return QB_EUNSUPPORTED;
  if (N == 0) return QB_OK;
  if (batch_tokens == 0 || batch_tokens > N) batch_tokens = N;
  if (N > INT32_MAX) return QB_EOVERFLOW;
  return launch_lei_apply_overlap(grad, N, E, batch_tokens, workspace, as_stream(stream));
}

int qb_router_gemm(const void* hidden, const void* w_t, int64_t M, int H, int E, float* logits_out,
                   void* stream) {
  if (!hidden || !w_t || !logits_out) return QB_EINVAL;
  if (!aligned16(hidden) || !aligned16(w_t) || !aligned16(logits_out)) return QB_EINVAL;
  if (M < 0) return QB_EINVAL;
  if (M > INT32_MAX) return QB_EOVERFLOW;
  if (E < 32 || E > 256 || E % 32 != 0 || H < 64 || H % 64 != 0) return QB_EUNSUPPORTED;
  if (M == 0) return QB_OK;
  return launch_router_gemm(hidden, w_t, M, H, E, logits_out, as_stream(stream));
}

int qb_router_gemm_hist_hi(const void* hidden, const void* w_t, int64_t M, int H, int E, int k,
                           const float* bias, float* logits_out, int32_t* hist_hi,
                           uint16_t* keys_out, int32_t* topk_out, float* alpha_out,
                           void* stream) {
  return router_gemm_hist_hi(hidden, w_t, M, H, E, k, bias, logits_out, hist_hi, keys_out,
                             topk_out, alpha_out, stream, false);
}

int qb_router_gemm_hist_hi_next(const void* hidden, const void* w_t, int64_t M, int H, int E,
                                int k, const float* bias, float* logits_out, int32_t* hist_hi,
                                uint16_t* keys_out, int32_t* topk_out, float* alpha_out,
                                void* stream) {
  return router_gemm_hist_hi(hidden, w_t, M, H, E, k, bias, logits_out, hist_hi, keys_out,
                             topk_out, alpha_out, stream, true);
}

int qb_rank_average(const uint16_t* qkeys, int P, int E, float* bias_out, void* stream) {
  if (!qkeys || !bias_out || P < 1) return QB_EINVAL;
  if (!supported_E(E)) return QB_EUNSUPPORTED;
  return launch_rank_average(qkeys, P, E, bias_out, as_stream(stream));
}

int qb_maxvio(const int32_t* topk_idx, int64_t N, int E, int k, int64_t batch_tokens,
              int32_t* loads_out, double* maxvio_out, void* stream) {
  if (!topk_idx || !loads_out || !maxvio_out) return QB_EINVAL;
  if (!aligned16(topk_idx)) return QB_EINVAL;
  if (N < 1 || batch_tokens < 0) return QB_EINVAL;
  if (!supported_E(E)) return QB_EUNSUPPORTED;
  if (k < 1 || k >= E) return QB_EINVAL;
  if (batch_tokens == 0 || batch_tokens > N) batch_tokens = N;
  if (N > INT32_MAX) return QB_EOVERFLOW;
  return launch_maxvio(topk_idx, N, E, k, batch_tokens, loads_out, maxvio_out,
                       as_stream(stream));
}

int64_t qb_balance_workspace(int64_t N, int E, int64_t batch_tokens) {
  if (N < 0 || batch_tokens < 0) return QB_EINVAL;
  if (N > INT32_MAX) return QB_EOVERFLOW;
  if (!supported_E(E)) return QB_EUNSUPPORTED;
  if (N == 0) return 0;
  if (batch_tokens == 0 || batch_tokens > N) batch_tokens = N;
  return balance_workspace_bytes(N, E, batch_tokens);
}

int qb_balance_loss(const void* logits, int dtype, const int32_t* topk_idx,
                    const uint8_t* token_mask, int64_t N, int E, int k, int64_t batch_tokens,
                    int score, float coeff, int32_t* counts, int32_t* tokens, float* prob_sum,
                    float* loss, void* workspace, int64_t workspace_bytes, void* stream) {
  const int st = check_balance_args(logits, dtype, N, E, k, batch_tokens, score);
  if (st != QB_OK || N == 0) return st;
  if (!topk_idx || !counts || !tokens || !prob_sum || !loss) return QB_EINVAL;
  if (!aligned4(topk_idx) || !aligned4(counts) || !aligned4(tokens) || !aligned4(prob_sum) ||
      !aligned4(loss))
    return QB_EINVAL;
  if (batch_tokens == 0 || batch_tokens > N) batch_tokens = N;
  const int64_t need = balance_workspace_bytes(N, E, batch_tokens);
  if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need))
    return QB_EINVAL;
  return launch_balance_loss(logits, dtype, topk_idx, token_mask, N, E, k, batch_tokens, score,
                             coeff, counts, tokens, prob_sum, loss, workspace, as_stream(stream));
}

int qb_balance_grad(const void* logits, int dtype, const uint8_t* token_mask,
                    const int32_t* counts, const int32_t* tokens, const float* loss_grad,
                    int64_t N, int E, int k, int64_t batch_tokens, int score, float coeff,
                    float* grad, int accumulate, void* stream) {
  const int st = check_balance_args(logits, dtype, N, E, k, batch_tokens, score);
  if (st != QB_OK || N == 0) return st;
  if (!counts || !tokens || !loss_grad || !grad || !aligned16(grad)) return QB_EINVAL;
  if (!aligned4(counts) || !aligned4(tokens) || !aligned4(loss_grad)) return QB_EINVAL;
  if (batch_tokens == 0 || batch_tokens > N) batch_tokens = N;
  return launch_balance_grad(logits, dtype, token_mask, counts, tokens, loss_grad, N, E, k,
                             batch_tokens, score, coeff, grad, accumulate, as_stream(stream));
}

int64_t qb_order_workspace(int64_t N, int E, int k) {
  if (N < 0 || k < 1) return QB_EINVAL;
  if (!supported_E(E)) return QB_EUNSUPPORTED;
  if (N > INT32_MAX / k) return QB_EOVERFLOW;
  return order_workspace_bytes(N, E, k);
}

int qb_expert_order(const int32_t* topk_idx, int64_t N, int E, int k, int32_t* counts,
                    int32_t* offsets, int32_t* slot_of, int32_t* token_of, void* workspace,
                    int64_t workspace_bytes, void* stream) {
  if (!counts || !offsets || N < 0 || k < 1) return QB_EINVAL;
  if (!supported_E(E)) return QB_EUNSUPPORTED;
  if (N > INT32_MAX / k) return QB_EOVERFLOW;
  if (N > 0 && (!topk_idx || !slot_of || !token_of || !workspace)) return QB_EINVAL;
  if (!aligned4(topk_idx) || !aligned4(counts) || !aligned4(offsets) || !aligned4(slot_of) ||
      !aligned4(token_of) || !aligned16(workspace))
    return QB_EINVAL;
  if (workspace_bytes < order_workspace_bytes(N, E, k)) return QB_EINVAL;
  return launch_expert_order(topk_idx, N, E, k, counts, offsets, slot_of, token_of, workspace,
                             as_stream(stream));
}

int64_t qb_fp8_scale_pitch(int64_t n) { return n < 0 ? (int64_t)QB_EINVAL : fp8_scale_pitch(n); }

int64_t qb_fp8_cols_width(int64_t M, int G) {
  if (M < 0 || G < 1) return QB_EINVAL;
  return (M + 127 * (int64_t)G) / 128 * 128;
}

int qb_fp8_quantize_rows(const void* x, int dtype, int64_t x_rows, int64_t ld,
                         const int32_t* row_idx, int64_t M, int K, uint8_t* q, uint8_t* scale,
                         void* stream) {
  const int st = check_source(x, dtype, x_rows, ld, row_idx, M, K);
  if (st != QB_OK) return st;
  if (K > 512 * 65535) return QB_EOVERFLOW;  // a grid row for each 512 columns
  if (M == 0) return QB_OK;
  if (!q || !scale || !aligned16(q) || !aligned16(scale)) return QB_EINVAL;
  return launch_fp8_rows(x, dtype, x_rows, ld, row_idx, M, K, q, scale, as_stream(stream));
}

int qb_fp8_quantize_cols(const void* x, int dtype, int64_t x_rows, int64_t ld,
                         const int32_t* row_idx, const int32_t* offsets, int G, int64_t M, int K,
                         int64_t width, uint8_t* q_t, uint8_t* scale_t, void* stream) {
  int st = check_source(x, dtype, x_rows, ld, row_idx, M, K);
  if (st != QB_OK) return st;
  st = check_groups(offsets, G, M);
  if (st != QB_OK) return st;
  if (width % 128 != 0 || width < qb_fp8_cols_width(M, G)) return QB_EINVAL;
  if (width > INT32_MAX) return QB_EOVERFLOW;
  if (width == 0) return QB_OK;
  if (!q_t || !scale_t || !aligned16(q_t) || !aligned16(scale_t)) return QB_EINVAL;
  if ((int64_t)((K + 127) / 128) * ((width + 511) / 512) > INT32_MAX) return QB_EOVERFLOW;
  return launch_fp8_cols(x, dtype, x_rows, ld, row_idx, offsets, G, M, K, width, q_t, scale_t,
                         as_stream(stream));
}

int qb_fp8_quantize_blocks(const void* w, int dtype, int G, int N, int K, uint8_t* q,
                           uint8_t* scale, uint8_t* q_t, uint8_t* scale_t, void* stream) {
  if (!w || !q || !scale || !is_dtype(dtype)) return QB_EINVAL;
  if (!q_t != !scale_t) return QB_EINVAL;
  if (!aligned16(w) || !aligned16(q) || !aligned16(scale) || !aligned16(q_t) ||
      !aligned16(scale_t))
    return QB_EINVAL;
  if (G < 1 || N < 1 || K < 16 || K % 16 != 0 || (q_t && N % 16 != 0)) return QB_EINVAL;
  if ((int64_t)((K + 127) / 128) * ((N + 127) / 128) > INT32_MAX / G) return QB_EOVERFLOW;
  return launch_fp8_blocks(w, dtype, G, N, K, q, scale, q_t, scale_t, as_stream(stream));
}

int qb_fp8_expert_gemm(const uint8_t* a, const uint8_t* a_scale, const uint8_t* b,
                       const uint8_t* b_scale, const int32_t* offsets, int G, int64_t M, int N,
                       int K, void* out, int out_dtype, void* stream) {
  if (!b || !b_scale || !is_dtype(out_dtype)) return QB_EINVAL;
  if (M > 0 && (!a || !a_scale || !out)) return QB_EINVAL;
  if (!aligned16(a) || !aligned16(a_scale) || !aligned16(b) || !aligned16(b_scale) ||
      !aligned16(out))
    return QB_EINVAL;
  const int st = check_groups(offsets, G, M);
  if (st != QB_OK) return st;
  if (N < 1 || K < 16 || K % 16 != 0) return QB_EINVAL;
  if ((int64_t)N > INT32_MAX - 256 || (int64_t)K > INT32_MAX - 256) return QB_EOVERFLOW;
  if (M == 0) return QB_OK;
  return launch_fp8_expert_gemm(a, a_scale, b, b_scale, offsets, G, M, N, K, out, out_dtype,
                                as_stream(stream));
}

int qb_fp8_expert_wgrad(const uint8_t* a_t, const uint8_t* a_scale, const uint8_t* b_t,
                        const uint8_t* b_scale, const int32_t* offsets, int G, int64_t width,
                        int N, int K, void* out, int out_dtype, int accumulate, void* stream) {
  // no tokens, no addresses: empty operands have none
  if (width != 0 && (!a_t || !a_scale || !b_t || !b_scale)) return QB_EINVAL;
  if (!out || !is_dtype(out_dtype)) return QB_EINVAL;
  if (!aligned16(a_t) || !aligned16(a_scale) || !aligned16(b_t) || !aligned16(b_scale) ||
      !aligned16(out))
    return QB_EINVAL;
  const int st = check_groups(offsets, G, width);
  if (st != QB_OK) return st;
  if (N < 1 || K < 1 || (accumulate && out_dtype != QB_F32)) return QB_EINVAL;
  if (N > INT32_MAX - 256 || K > INT32_MAX - 256) return QB_EOVERFLOW;
  // one group without tokens has no columns (qb_fp8_cols_width); several have some always
  if (width == 0 && G == 1)
    return launch_no_wgrad(N, K, out, out_dtype, accumulate, as_stream(stream));
  if (width < 128 || width % 128 != 0) return QB_EINVAL;
  return launch_fp8_expert_wgrad(a_t, a_scale, b_t, b_scale, offsets, G, width, N, K, out,
                                 out_dtype, accumulate, as_stream(stream));
}

int qb_device_status(int* flags_out) {
  int* p = device_status_ptr();
  if (!p) return QB_ECUDA;
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_status_word, sizeof(int)) != cudaSuccess) return QB_ECUDA;
  const int zero = 0;
  if (cudaMemcpyToSymbol(g_status_word, &zero, sizeof(int)) != cudaSuccess) return QB_ECUDA;
  if (flags_out) *flags_out = v;
  return v ? QB_EDEVICE : QB_OK;
}

}  // extern "C"
