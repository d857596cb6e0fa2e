// Host-side interface between the C ABI of the training-step operators
// (step_abi.cu) and their kernels: the residual update with its norms, the
// token embedding, the vocabulary cross entropy, gradient clipping.
#pragma once
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "internal.h"

namespace moe {

// Raises a kernel's dynamic shared-memory limit, once per device.
template <typename K>
inline cudaError_t allow_smem(K kern, std::atomic<unsigned long long>& devices, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (devices.load(std::memory_order_acquire) >> dev & 1) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) devices.fetch_or(1ull << dev, std::memory_order_release);
  return e;
}

inline size_t up256(size_t b) { return (b + 255) & ~size_t(255); }

// ------------------------------------------------------------ residual + norms
constexpr int kNormMaxD = 8192;
constexpr int kNormSms = 152;  // the backward's grid, and with it its workspace, is sized for the 152-SM part

struct NormArgs {
  const void* r;        // [T, d] bf16 or fp32, nullable
  const void* o;        // [T, d] bf16, nullable
  const float* gate;    // [T] or [d]
  int gate_kind;        // MOE_GATE_*
  const void* w_post;   // [d] bf16, nullable
  const void* w_pre;    // [d] bf16 (with x)
  int T, d;
  float alpha, eps;
  void* r_out;          // [T, d], nullable
  void* x;              // [T, d] bf16, nullable
  float* rstd_post;     // [T], nullable
  float* rstd_pre;
};
cudaError_t launch_residual_norm(const NormArgs& a, bool r_f32, cudaStream_t s);

struct NormBwdArgs {
  const void* dx;       // [T, d] bf16, nullable
  const void* dr_out;   // [T, d] like r, nullable
  const void* o;        // [T, d] bf16, nullable
  const float* gate;
  int gate_kind;
  const void* w_post;
  const void* w_pre;
  const void* r_out;    // [T, d] (with dx)
  const float* rstd_post;
  const float* rstd_pre;
  int T, d;
  float alpha;
  void* dr;             // [T, d] like r, nullable
  void* d_o;            // [T, d] bf16 (with o)
  float* dgate;         // [T] or [d]
  float* dw_post;       // [d]
  float* dw_pre;        // [d]
  float* part;          // workspace: [CTAs][2][d]
  int* status;
};
size_t residual_norm_ws_bytes(int T, int d);
cudaError_t launch_residual_norm_bwd(const NormBwdArgs& a, bool r_f32, cudaStream_t s);

// ------------------------------------------------------------ token embedding
cudaError_t launch_embedding(const void* table, const int32_t* ids, int T, int V, int d, float scale, void* out,
                             int* status, cudaStream_t s);
// what T tokens need, and the most that any batch of up to T tokens does
size_t embedding_ws_bytes(int T, int d);
size_t embedding_ws_bytes_up_to(int T, int d);
cudaError_t launch_embedding_bwd(const void* dout, const int32_t* ids, int T, int V, int d, float scale,
                                 bool accumulate, void* dtable, void* ws, int* status, cudaStream_t s);

// ------------------------------------------------------------ gradient clipping
size_t grad_clip_ws_bytes(long long n_tensors);
// grads, outs (nullable: norm and coefficient only), sizes, types: host arrays
cudaError_t launch_grad_clip(const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* types,
                             int n, float max_norm, float* norm, float* coef, void* ws, int* status, cudaStream_t s);

// ------------------------------------------------------------ vocabulary cross entropy
struct VocabArgs {
  const void* x;           // [T, d] bf16
  const void* W;           // [V, d] bf16
  const int32_t* targets;  // [T]
  int T, d, V;
  float z_weight;
};
// columns of one piece of the backward (a multiple of 256, at most V rounded
// up): the caller's, or the default if it is 0
int vocab_piece(int T, int V, int piece);
size_t vocab_fwd_ws_bytes(int T, int d, int V);
size_t vocab_bwd_ws_bytes(int T, int d, int V, int piece);
// the most that any batch of up to T tokens needs
size_t vocab_fwd_ws_bytes_up_to(int T, int d, int V);
size_t vocab_bwd_ws_bytes_up_to(int T, int d, int V, int piece);
cudaError_t launch_cross_entropy(const VocabArgs& a, float* loss, float* lse, void* ws, int* status, cudaStream_t s);
// dx [T, d], dW [V, d] bf16, each nullable
cudaError_t launch_cross_entropy_bwd(const VocabArgs& a, const float* lse, const float* dloss, int piece, void* dx,
                                     void* dW, void* ws, int* status, cudaStream_t s);

}  // namespace moe
