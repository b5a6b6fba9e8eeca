// The C ABI of the scoring and distillation calls (declared in include/kdkl.h): argument
// checks, workspace layout and launches.  Host code only.
#include <math.h>

#include "kd_internal.h"

using namespace kd;

namespace {

constexpr int64_t kMaxV = int64_t(1) << 30;

// A step over up to this many rows lets each block count the valid ones, which up to here costs no
// more than a launch does (in blocks / ahead, us: 1024 x 1000 14.4 / 16.4, 8192 x 1000 45.1 / 45.0,
// 16384 x 1000 79.9 / 77.2, 131072 x 1000 584 / 549; 8192 x 4096 55.8 / 56.3, 16384 x 4096 105.1 /
// 103.8; 8192 x 32000 198 / 200, 32768 x 32000 737 / 739).
constexpr int64_t kCountInBlock = 8192;

size_t elt_size(int dtype) { return dtype == KD_F32 ? 4 : 2; }

// What every call on dense logits checks: sizes, type, temperature, alignment to the element.
kd_status check_logits(const void* z, int dtype, int64_t N, int64_t V, int64_t ld, float tau) {
  if (N < 1 || N > 0x7fffffffLL || V < 1 || V > kMaxV || ld < V) return KD_ERR_INVALID_ARG;
  if (dtype != KD_BF16 && dtype != KD_F16 && dtype != KD_F32) return KD_ERR_INVALID_ARG;
  if (!(tau > 0.f) || !isfinite(tau)) return KD_ERR_INVALID_ARG;
  if (!z || !aligned(z, elt_size(dtype))) return KD_ERR_INVALID_ARG;
  return KD_OK;
}

// The gradient matrix: its own, or the logits themselves.
kd_status check_grad(const void* z, int dtype, int64_t N, int64_t V, int64_t ld, const void* g, int64_t ld_g) {
  if (!g || !aligned(g, elt_size(dtype)) || ld_g < V) return KD_ERR_INVALID_ARG;
  if (g == z) return ld_g == ld ? KD_OK : KD_ERR_INVALID_ARG;
  const uintptr_t a = reinterpret_cast<uintptr_t>(z), b = reinterpret_cast<uintptr_t>(g);
  const size_t na = (size_t(N - 1) * size_t(ld) + size_t(V)) * elt_size(dtype);
  const size_t nb = (size_t(N - 1) * size_t(ld_g) + size_t(V)) * elt_size(dtype);
  return (a + na <= b || b + nb <= a) ? KD_OK : KD_ERR_INVALID_ARG;
}

bool ok4(const void* p) { return p != nullptr && aligned(p, 4); }
bool ok4_or_null(const void* p) { return p == nullptr || aligned(p, 4); }

kd_status check_ws(const void* ws, size_t have, size_t need) {
  return (ws && aligned(ws, 256) && have >= need) ? KD_OK : KD_ERR_WORKSPACE;
}

// The block that holds the error word: the workspace's own, or the caller's.
kd_status check_control(const void* control) {
  return (control && aligned(control, 256)) ? KD_OK : KD_ERR_WORKSPACE;
}

size_t logits_kl_ws(int64_t N) { return sizeof(Ctrl) + align_up(size_t(N) * 4, 256); }

kd_status check_teacher(const int32_t* ids, const float* tlog, int K, const float* t_lse, int64_t V, int dtype) {
  if (K < 1 || K > KD_MAX_K || int64_t(K) > V) return KD_ERR_INVALID_ARG;
  if (!ok4(ids) || !ok4(tlog) || !ok4_or_null(t_lse)) return KD_ERR_INVALID_ARG;
  return logits_kl_fits(V, K, dtype) ? KD_OK : KD_ERR_UNSUPPORTED;
}

// Valid positions: counted on the device where there is a mask (NULL: all N are).
kd_status count_valid(const uint8_t* mask, int64_t N, Ctrl* ctrl, const int32_t** n_valid, cudaStream_t s) {
  *n_valid = mask ? &ctrl->n_valid : nullptr;
  return mask ? map_cuda(launch_count_valid(mask, N, &ctrl->n_valid, s)) : KD_OK;
}

}  // namespace

extern "C" {

int kd_workspace_clear(void* ws, size_t ws_bytes, void* stream) {
  kd_status st = check_ws(ws, ws_bytes, sizeof(Ctrl));
  if (st != KD_OK) return st;
  return map_cuda(cudaMemsetAsync(ws, 0, sizeof(Ctrl), static_cast<cudaStream_t>(stream)));
}

size_t kd_token_logprobs_workspace(int64_t N, int64_t V) {
  (void)N;
  (void)V;
  return sizeof(Ctrl);
}

int kd_token_logprobs_fwd(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld, const int32_t* tokens,
                          int M, const uint8_t* mask, float tau, int top, float* logp_out, float* lse_out,
                          float* entropy_out, int32_t* top_ids_out, float* top_logp_out, void* ws, size_t ws_bytes,
                          void* stream) {
  kd_status st = check_logits(logits, dtype, N, V, ld, tau);
  if (st != KD_OK) return st;
  if (M < 1 || M > KD_MAX_K || top < 0 || top > KD_MAX_TOP || int64_t(top) > V) return KD_ERR_INVALID_ARG;
  if (!ok4(tokens) || !ok4(logp_out) || !ok4(lse_out) || !ok4_or_null(entropy_out)) return KD_ERR_INVALID_ARG;
  if (top > 0 ? !(ok4(top_ids_out) && ok4(top_logp_out)) : (top_ids_out || top_logp_out)) return KD_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, kd_token_logprobs_workspace(N, V))) != KD_OK) return st;
  if ((st = check_device()) != KD_OK) return st;
  return map_cuda(launch_logprobs_fwd(logits, dtype, N, V, ld, tokens, M, mask, tau, top, logp_out, lse_out,
                                      entropy_out, top_ids_out, top_logp_out, &static_cast<Ctrl*>(ws)->err,
                                      static_cast<cudaStream_t>(stream)));
}

int kd_token_logprobs_bwd(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld, const int32_t* tokens,
                          int M, const uint8_t* mask, float tau, const float* lse, const float* entropy,
                          const float* grad_logp, const float* grad_entropy, void* grad_logits, int64_t ld_grad,
                          void* ws, size_t ws_bytes, void* stream) {
  kd_status st = check_logits(logits, dtype, N, V, ld, tau);
  if (st != KD_OK) return st;
  if (M < 1 || M > KD_MAX_K) return KD_ERR_INVALID_ARG;
  if (!ok4(tokens) || !ok4(lse) || !ok4(grad_logp) || !ok4_or_null(grad_entropy) || !ok4_or_null(entropy) ||
      (grad_entropy && !entropy))
    return KD_ERR_INVALID_ARG;
  if ((st = check_grad(logits, dtype, N, V, ld, grad_logits, ld_grad)) != KD_OK) return st;
  if ((st = check_ws(ws, ws_bytes, kd_token_logprobs_workspace(N, V))) != KD_OK) return st;
  if ((st = check_device()) != KD_OK) return st;
  return map_cuda(launch_logprobs_bwd(logits, dtype, N, V, ld, tokens, M, mask, tau, lse, entropy, grad_logp,
                                      grad_entropy, grad_logits, ld_grad, &static_cast<Ctrl*>(ws)->err,
                                      static_cast<cudaStream_t>(stream)));
}

size_t kd_logits_kl_workspace(int64_t N, int64_t V, int K) {
  (void)V;
  (void)K;
  return N < 1 ? sizeof(Ctrl) : logits_kl_ws(N);
}

int kd_logits_kl_fwd(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld, const int32_t* t_ids,
                     const float* t_logits, int K, const float* t_lse, const uint8_t* mask, float tau,
                     float* loss_out, float* stats_out, float* kl_per_token_out, void* ws, size_t ws_bytes,
                     void* stream) {
  return kd_logits_kl_fwd_ctl(logits, dtype, N, V, ld, t_ids, t_logits, K, t_lse, mask, tau, loss_out, stats_out,
                              kl_per_token_out, ws, ws_bytes, ws, stream);
}

int kd_logits_kl_fwd_ctl(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld, const int32_t* t_ids,
                         const float* t_logits, int K, const float* t_lse, const uint8_t* mask, float tau,
                         float* loss_out, float* stats_out, float* kl_per_token_out, void* ws, size_t ws_bytes,
                         void* control, void* stream) {
  kd_status st = check_logits(logits, dtype, N, V, ld, tau);
  if (st != KD_OK) return st;
  if ((st = check_teacher(t_ids, t_logits, K, t_lse, V, dtype)) != KD_OK) return st;
  if (!ok4(loss_out) || !stats_out || !aligned(stats_out, 16) || !ok4_or_null(kl_per_token_out))
    return KD_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, logits_kl_ws(N))) != KD_OK) return st;
  if ((st = check_control(control)) != KD_OK) return st;
  if ((st = check_device()) != KD_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* kl = kl_per_token_out ? kl_per_token_out : reinterpret_cast<float*>(static_cast<Ctrl*>(ws) + 1);
  if (launch_logits_kl(1, logits, dtype, N, V, ld, t_ids, t_logits, K, t_lse, mask, tau, stats_out, kl, nullptr,
                       nullptr, nullptr, 0, &static_cast<Ctrl*>(control)->err, s) != cudaSuccess)
    return KD_ERR_CUDA;
  return map_cuda(launch_masked_mean(kl, mask, N, loss_out, s));
}

int kd_logits_kl_bwd(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld, const int32_t* t_ids,
                     const float* t_logits, int K, const float* t_lse, const uint8_t* mask, float tau,
                     const float* stats, const float* grad_loss, void* grad_logits, int64_t ld_grad, void* ws,
                     size_t ws_bytes, void* stream) {
  return kd_logits_kl_bwd_ctl(logits, dtype, N, V, ld, t_ids, t_logits, K, t_lse, mask, tau, stats, grad_loss,
                              grad_logits, ld_grad, ws, ws_bytes, ws, stream);
}

int kd_logits_kl_bwd_ctl(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld, const int32_t* t_ids,
                         const float* t_logits, int K, const float* t_lse, const uint8_t* mask, float tau,
                         const float* stats, const float* grad_loss, void* grad_logits, int64_t ld_grad, void* ws,
                         size_t ws_bytes, void* control, void* stream) {
  kd_status st = check_logits(logits, dtype, N, V, ld, tau);
  if (st != KD_OK) return st;
  if ((st = check_teacher(t_ids, t_logits, K, t_lse, V, dtype)) != KD_OK) return st;
  if (!stats || !aligned(stats, 16) || !ok4(grad_loss)) return KD_ERR_INVALID_ARG;
  if ((st = check_grad(logits, dtype, N, V, ld, grad_logits, ld_grad)) != KD_OK) return st;
  if ((st = check_ws(ws, ws_bytes, logits_kl_ws(N))) != KD_OK) return st;
  if ((st = check_control(control)) != KD_OK) return st;
  if ((st = check_device()) != KD_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int32_t* n_valid;
  if ((st = count_valid(mask, N, static_cast<Ctrl*>(ws), &n_valid, s)) != KD_OK) return st;
  return map_cuda(launch_logits_kl(2, logits, dtype, N, V, ld, t_ids, t_logits, K, t_lse, mask, tau,
                                   const_cast<float*>(stats), nullptr, grad_loss, n_valid, grad_logits, ld_grad,
                                   &static_cast<Ctrl*>(control)->err, s));
}

int kd_logits_kl_step(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld, const int32_t* t_ids,
                      const float* t_logits, int K, const float* t_lse, const uint8_t* mask, float tau,
                      const float* grad_loss, float* loss_out, float* kl_per_token_out, void* grad_logits,
                      int64_t ld_grad, void* ws, size_t ws_bytes, void* stream) {
  return kd_logits_kl_step_ctl(logits, dtype, N, V, ld, t_ids, t_logits, K, t_lse, mask, tau, grad_loss, loss_out,
                               kl_per_token_out, grad_logits, ld_grad, ws, ws_bytes, ws, stream);
}

int kd_logits_kl_step_ctl(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld, const int32_t* t_ids,
                          const float* t_logits, int K, const float* t_lse, const uint8_t* mask, float tau,
                          const float* grad_loss, float* loss_out, float* kl_per_token_out, void* grad_logits,
                          int64_t ld_grad, void* ws, size_t ws_bytes, void* control, void* stream) {
  kd_status st = check_logits(logits, dtype, N, V, ld, tau);
  if (st != KD_OK) return st;
  if ((st = check_teacher(t_ids, t_logits, K, t_lse, V, dtype)) != KD_OK) return st;
  if (!ok4(loss_out) || !ok4(grad_loss) || !ok4_or_null(kl_per_token_out)) return KD_ERR_INVALID_ARG;
  if ((st = check_grad(logits, dtype, N, V, ld, grad_logits, ld_grad)) != KD_OK) return st;
  if ((st = check_ws(ws, ws_bytes, logits_kl_ws(N))) != KD_OK) return st;
  if ((st = check_control(control)) != KD_OK) return st;
  if ((st = check_device()) != KD_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Ctrl* ctrl = static_cast<Ctrl*>(ws);
  float* kl = kl_per_token_out ? kl_per_token_out : reinterpret_cast<float*>(ctrl + 1);
  const int32_t* n_valid = nullptr;
  if (N > kCountInBlock && (st = count_valid(mask, N, ctrl, &n_valid, s)) != KD_OK) return st;
  if (launch_logits_kl(3, logits, dtype, N, V, ld, t_ids, t_logits, K, t_lse, mask, tau, nullptr, kl, grad_loss,
                       n_valid, grad_logits, ld_grad, &static_cast<Ctrl*>(control)->err, s) != cudaSuccess)
    return KD_ERR_CUDA;
  return map_cuda(launch_masked_mean(kl, mask, N, loss_out, s));
}

}  // extern "C"
