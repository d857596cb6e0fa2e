// C ABI of the training-step operators (include/moe.h): argument checks on
// the host, then the launches.
#include "../../include/moe.h"
#include "step.h"

using namespace moe;

namespace {
int done(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  record_cuda_error(e);
  return MOE_ERR_CUDA;
}
cudaStream_t st(void* s) { return static_cast<cudaStream_t>(s); }
bool ws_ok(const void* ws) { return ws && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0; }
// every pointer of the list 16-byte aligned (NULL is)
template <typename... P>
bool all16(P... p) {
  return (al16(p) && ...);
}
int check_norm(int T, int d, int gate_kind) {
  if (T < 1 || d < 1 || gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_CHANNEL) return MOE_ERR_INVALID_ARG;
  if (d % 64 != 0 || d > kNormMaxD) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
int check_embedding(int T, int V, int d) {
  if (T < 1 || V < 1 || d < 1) return MOE_ERR_INVALID_ARG;
  if (d % 64 != 0 || d > 65536 || T > (1 << 30) || V > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
int check_vocab(int T, int d, int V) {
  if (T < 1 || d < 1 || V < 1) return MOE_ERR_INVALID_ARG;
  if (d % 64 != 0 || d > 65536 || T > (1 << 24) || V > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
}  // namespace

extern "C" {

int moe_residual_norm(const void* r, const void* o, const float* gate, int gate_kind, const void* w_post,
                      const void* w_pre, int T, int d, int r_f32, float alpha, float eps, void* r_out, void* x,
                      float* rstd_post, float* rstd_pre, void* stream) {
  int rc = check_norm(T, d, gate_kind);
  if (rc) return rc;
  if ((!r && !o) || (!r_out && !x) || (x == nullptr) != (w_pre == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!o && (gate_kind != MOE_GATE_NONE || w_post)) return MOE_ERR_INVALID_ARG;
  if ((gate_kind != MOE_GATE_NONE) != (gate != nullptr)) return MOE_ERR_INVALID_ARG;
  if ((rstd_post && !w_post) || (rstd_pre && !x)) return MOE_ERR_INVALID_ARG;
  if (!all16(r, o, gate_kind == MOE_GATE_CHANNEL ? gate : nullptr, w_post, w_pre, r_out, x)) return MOE_ERR_INVALID_ARG;
  NormArgs a{r, o, gate, gate_kind, w_post, w_pre, T, d, alpha, eps, r_out, x, rstd_post, rstd_pre};
  return done(launch_residual_norm(a, r_f32 != 0, st(stream)));
}

int moe_residual_norm_workspace(int T, int d, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  int rc = check_norm(T, d, MOE_GATE_NONE);
  if (rc) return rc;
  *bytes = residual_norm_ws_bytes(T, d);
  return MOE_OK;
}

int moe_residual_norm_bwd(const void* dx, const void* dr_out, const void* o, const float* gate, int gate_kind,
                          const void* w_post, const void* w_pre, const void* r_out, const float* rstd_post,
                          const float* rstd_pre, int T, int d, int r_f32, float alpha, void* dr, void* d_o,
                          float* dgate, float* dw_post, float* dw_pre, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_norm(T, d, gate_kind);
  if (rc) return rc;
  if (!dx && !dr_out) return MOE_ERR_INVALID_ARG;
  if (dx ? (!w_pre || !r_out || !rstd_pre) : dw_pre != nullptr) return MOE_ERR_INVALID_ARG;
  if ((o == nullptr) != (d_o == nullptr) || (!o && !dr)) return MOE_ERR_INVALID_ARG;
  if (!o && (gate_kind != MOE_GATE_NONE || w_post)) return MOE_ERR_INVALID_ARG;
  if ((gate_kind != MOE_GATE_NONE) != (gate != nullptr) || (dgate && !gate)) return MOE_ERR_INVALID_ARG;
  if (w_post ? !rstd_post : dw_post != nullptr) return MOE_ERR_INVALID_ARG;
  const bool channel = gate_kind == MOE_GATE_CHANNEL;
  if (!all16(dx, dr_out, o, channel ? gate : nullptr, w_post, w_pre, r_out, dr, d_o, dw_post, dw_pre,
             channel ? dgate : nullptr))
    return MOE_ERR_INVALID_ARG;
  if (ws && !ws_ok(ws)) return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < residual_norm_ws_bytes(T, d)) return MOE_ERR_WORKSPACE;
  NormBwdArgs a{dx, dr_out, o, gate, gate_kind, w_post, w_pre, r_out, rstd_post, rstd_pre, T, d, alpha, dr, d_o,
                dgate, dw_post, dw_pre, static_cast<float*>(ws), device_status_ptr()};
  return done(launch_residual_norm_bwd(a, r_f32 != 0, st(stream)));
}

int moe_embedding(const void* table, const int32_t* ids, int T, int V, int d, float scale, void* out, void* stream) {
  int rc = check_embedding(T, V, d);
  if (rc) return rc;
  if (!table || !ids || !out || !all16(table, out)) return MOE_ERR_INVALID_ARG;
  return done(launch_embedding(table, ids, T, V, d, scale, out, device_status_ptr(), st(stream)));
}

int moe_embedding_workspace(int T, int V, int d, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  int rc = check_embedding(T, V, d);
  if (rc) return rc;
  *bytes = embedding_ws_bytes_up_to(T, d);
  return MOE_OK;
}

int moe_embedding_bwd(const void* dout, const int32_t* ids, int T, int V, int d, float scale, int accumulate,
                      void* dtable, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_embedding(T, V, d);
  if (rc) return rc;
  if (!dout || !ids || !dtable || !all16(dout, dtable)) return MOE_ERR_INVALID_ARG;
  if (ws && !ws_ok(ws)) return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < embedding_ws_bytes(T, d)) return MOE_ERR_WORKSPACE;
  return done(launch_embedding_bwd(dout, ids, T, V, d, scale, accumulate != 0, dtable, ws, device_status_ptr(),
                                   st(stream)));
}

int moe_cross_entropy_workspace(int T, int d, int V, int piece, int grad, size_t* bytes) {
  if (!bytes || piece < 0) return MOE_ERR_INVALID_ARG;
  int rc = check_vocab(T, d, V);
  if (rc) return rc;
  size_t b = vocab_fwd_ws_bytes_up_to(T, d, V);
  const size_t g = grad ? vocab_bwd_ws_bytes_up_to(T, d, V, piece) : 0;
  *bytes = g > b ? g : b;
  return MOE_OK;
}

int moe_cross_entropy(const void* x, const void* W, const int32_t* targets, int T, int d, int V, float z_weight,
                      float* loss, float* lse, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_vocab(T, d, V);
  if (rc) return rc;
  if (!x || !W || !targets || !loss || !lse || !all16(x, W)) return MOE_ERR_INVALID_ARG;
  if (ws && !ws_ok(ws)) return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < vocab_fwd_ws_bytes(T, d, V)) return MOE_ERR_WORKSPACE;
  const VocabArgs a{x, W, targets, T, d, V, z_weight};
  return done(launch_cross_entropy(a, loss, lse, ws, device_status_ptr(), st(stream)));
}

int moe_cross_entropy_bwd(const void* x, const void* W, const int32_t* targets, const float* lse, const float* dloss,
                          int T, int d, int V, float z_weight, int piece, void* dx, void* dW, void* ws,
                          size_t ws_bytes, void* stream) {
  int rc = check_vocab(T, d, V);
  if (rc) return rc;
  if (!x || !W || !targets || !lse || !dloss || (!dx && !dW) || piece < 0) return MOE_ERR_INVALID_ARG;
  if (!all16(x, W, dx, dW)) return MOE_ERR_INVALID_ARG;
  if (ws && !ws_ok(ws)) return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < vocab_bwd_ws_bytes(T, d, V, piece)) return MOE_ERR_WORKSPACE;
  const VocabArgs a{x, W, targets, T, d, V, z_weight};
  return done(launch_cross_entropy_bwd(a, lse, dloss, piece, dx, dW, ws, device_status_ptr(), st(stream)));
}

int moe_grad_clip_workspace(int n, size_t* bytes) {
  if (!bytes || n < 1) return MOE_ERR_INVALID_ARG;
  *bytes = grad_clip_ws_bytes(n);
  return MOE_OK;
}

int moe_grad_clip(const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* types, int n,
                  float max_norm, float* norm, float* coef, void* ws, size_t ws_bytes, void* stream) {
  if (!grads || !sizes || !types || n < 1 || !norm) return MOE_ERR_INVALID_ARG;
  if (!(max_norm >= 0.0f)) return MOE_ERR_INVALID_ARG;  // NaN too
  for (int i = 0; i < n; ++i) {
    if (types[i] < MOE_GRAD_BF16 || types[i] > MOE_GRAD_F16 || sizes[i] < 0 || sizes[i] > (1LL << 40))
      return MOE_ERR_INVALID_ARG;
    const uintptr_t mask = types[i] == MOE_GRAD_F32 ? 3u : 1u;
    if (sizes[i] && (!grads[i] || (outs && !outs[i]))) return MOE_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(grads[i]) & mask) || (outs && (reinterpret_cast<uintptr_t>(outs[i]) & mask)))
      return MOE_ERR_INVALID_ARG;
  }
  if (ws && !ws_ok(ws)) return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < grad_clip_ws_bytes(n)) return MOE_ERR_WORKSPACE;
  return done(launch_grad_clip(grads, outs, sizes, types, n, max_norm, norm, coef, ws, device_status_ptr(),
                               st(stream)));
}

}  // extern "C"
