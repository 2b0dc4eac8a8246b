// qb_internal.h -- host-side helpers shared by the libqb translation units.
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/qb.h"

namespace qb {

// Device pointer to the library's device status word for the current device
// (set up on first use per device); nullptr if CUDA fails.
int* device_status_ptr();

// Streaming multiprocessor count of the current device (cached per device).
int sm_count();

inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Expert counts the kernels take: multiples of 32 from 32 to kMaxE.
constexpr int kMaxE = 1024;
inline bool supported_E(int E) { return E >= 32 && E <= kMaxE && E % 32 == 0; }

inline int launch_status() {
  return cudaPeekAtLastError() == cudaSuccess ? QB_OK : (cudaGetLastError(), QB_ECUDA);
}

// Raises a kernel's dynamic shared-memory limit, once per device (`done` holds
// a bit for each of the first 64).
template <class F>
bool smem_attribute(F kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load() & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
      cudaSuccess)
    return false;
  done.fetch_or(bit);
  return true;
}

// 8-bit operands: bytes of one row of scales (one byte for each 128 values,
// whole 32-bit words), and the most groups an offsets array describes.
inline int64_t fp8_scale_pitch(int64_t K) { return ((K + 127) / 128 + 3) / 4 * 4; }
constexpr int kMaxGroups = 1024;

// Launchers implemented in the kernel translation units.
int launch_route_hi(const void* logits, int dtype, const float* bias, int64_t N, int E, int k,
                    int32_t* hist, uint16_t* keys_out, int32_t* topk_out, float* alpha_out,
                    const int32_t* sel, const float* bounds, int nbins, cudaStream_t stream);
int launch_route_lo(const void* logits, int dtype, const float* bias, int64_t N, int E, int k,
                    int32_t* hist, uint16_t* keys_out, int32_t* topk_out, float* alpha_out,
                    const int32_t* sel, const float* bounds, int nbins, cudaStream_t stream);
int launch_route_k3(const void* logits, int dtype, const float* bias, int64_t N, int E, int k,
                    int32_t* hist, uint16_t* keys_out, int32_t* topk_out, float* alpha_out,
                    const int32_t* sel, const float* bounds, int nbins, cudaStream_t stream);
// EQB hi pass specialised to E = 256 (qb_route256.cuh), per input type;
// chained: a further microbatch right after another such call on the stream
// (qb_route_hist_hi_next).
int launch_route256_hi_f32(const void* logits, const float* bias, int64_t N, int k,
                           int32_t* hist, uint16_t* keys_out, int32_t* topk_out,
                           float* alpha_out, cudaStream_t stream, bool chained = false);
int launch_route256_hi_bf16(const void* logits, const float* bias, int64_t N, int k,
                            int32_t* hist, uint16_t* keys_out, int32_t* topk_out,
                            float* alpha_out, cudaStream_t stream, bool chained = false);
// alpha per token only (the first half of the K3 pass), E = 256; chained: a
// further microbatch right after another K3 call on the stream
// (k3_route_hist_next).
int launch_route256_alpha_f32(const void* logits, const float* bias, int64_t N, int k,
                              float* alpha_out, cudaStream_t stream, bool chained = false);
int launch_route256_alpha_bf16(const void* logits, const float* bias, int64_t N, int k,
                               float* alpha_out, cudaStream_t stream, bool chained = false);
int launch_keys_hist_lo(const uint16_t* keys, int64_t N, int E, const int32_t* sel,
                        int32_t* hist_lo, cudaStream_t stream);
int launch_select_hi(const int32_t* hist_hi, int E, int64_t r, int32_t* sel, int32_t* r_lo,
                     cudaStream_t stream);
int launch_finalize(int32_t* hist_hi, int32_t* hist_lo, const int32_t* sel, const int32_t* r_lo,
                    int E, float* bias_out, uint16_t* qkey_out, int reset, cudaStream_t stream);
int launch_k3_finalize(int32_t* hist, int E, int nbins, int64_t r, float* bounds,
                       float* bias_out, int reset, cudaStream_t stream);
int launch_k3_count(const void* logits, int dtype, const float* alpha, int64_t N, int E,
                    const float* bounds, int nbins, int32_t* hist, cudaStream_t stream);
int launch_zero_i32(int32_t* p, int64_t n, cudaStream_t stream);
int launch_wait_timeout_selftest(uint32_t polls, cudaStream_t stream);
int launch_router_gemm_route(const void* hidden, const void* w_t, int64_t M, int K, int k,
                             const float* bias, int32_t* hist, uint16_t* keys_out,
                             int32_t* topk_out, float* alpha_out, float* logits_out,
                             cudaStream_t stream, bool chained = false);
int launch_rank_average(const uint16_t* qkeys, int P, int E, float* bias_out,
                        cudaStream_t stream);
int launch_maxvio(const int32_t* topk, int64_t N, int E, int k, int64_t batch_tokens,
                  int32_t* loads, double* out, cudaStream_t stream);
int launch_sigmoid(const float* x, float* s, int64_t n, int scalar, cudaStream_t stream);
int launch_lei(float* grad, const int32_t* topk, int64_t N, int E, int k, float eta,
               int64_t batch_tokens, float* workspace, cudaStream_t stream);
int launch_lei_rho(const int32_t* topk, int64_t N, int E, int k, float eta,
                   int64_t batch_tokens, float* workspace, cudaStream_t stream);
int launch_lei_apply(float* grad, int64_t N, int E, int64_t batch_tokens, const float* workspace,
                     cudaStream_t stream);
int launch_lei_apply_overlap(float* grad, int64_t N, int E, int64_t batch_tokens,
                             const float* workspace, cudaStream_t stream);

int launch_router_gemm(const void* hidden, const void* w_t, int64_t M, int K, int E,
                       float* logits, cudaStream_t stream);

int launch_balance_loss(const void* logits, int dtype, const int32_t* topk, const uint8_t* mask,
                        int64_t N, int E, int k, int64_t batch_tokens, int score, float coeff,
                        int32_t* counts, int32_t* tokens, float* prob_sum, float* loss,
                        void* workspace, cudaStream_t stream);
int64_t balance_workspace_bytes(int64_t N, int E, int64_t batch_tokens);
int launch_balance_grad(const void* logits, int dtype, const uint8_t* mask, const int32_t* counts,
                        const int32_t* tokens, const float* loss_grad, int64_t N, int E, int k,
                        int64_t batch_tokens, int score, float coeff, float* grad, int accumulate,
                        cudaStream_t stream);
int64_t order_workspace_bytes(int64_t N, int E, int k);
int launch_expert_order(const int32_t* topk, int64_t N, int E, int k, int32_t* counts,
                        int32_t* offsets, int32_t* slot_of, int32_t* token_of, void* workspace,
                        cudaStream_t stream);
int launch_fp8_rows(const void* x, int dtype, int64_t x_rows, int64_t ld, const int32_t* row_idx,
                    int64_t M, int K, uint8_t* q, uint8_t* scale, cudaStream_t stream);
int launch_fp8_cols(const void* x, int dtype, int64_t x_rows, int64_t ld, const int32_t* row_idx,
                    const int32_t* offsets, int G, int64_t M, int K, int64_t width, uint8_t* q_t,
                    uint8_t* scale_t, cudaStream_t stream);
int launch_fp8_blocks(const void* w, int dtype, int G, int N, int K, uint8_t* q, uint8_t* scale,
                      uint8_t* q_t, uint8_t* scale_t, cudaStream_t stream);
int launch_fp8_expert_gemm(const void* a, const uint8_t* a_scale, const void* b,
                           const uint8_t* b_scale, const int32_t* offsets, int G, int64_t M, int N,
                           int K, void* out, int out_dtype, cudaStream_t stream);
int launch_fp8_expert_wgrad(const void* a_t, const uint8_t* a_scale, const void* b_t,
                            const uint8_t* b_scale, const int32_t* offsets, int G, int64_t width,
                            int N, int K, void* out, int out_dtype, int accumulate,
                            cudaStream_t stream);

enum RouteMode { kModeHi = 0, kModeLo = 1, kModeK3 = 2 };

}  // namespace qb
