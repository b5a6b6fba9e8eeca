// Launches of the KL on dense logits (kd_logits_kl.cuh) and the mean of its rows.
#include "kd_logits_kl.cuh"

namespace kd {

extern template cudaError_t lk_run<KD_BF16>(int, const LogitsKlArgs&, cudaStream_t);
extern template cudaError_t lk_run<KD_F16>(int, const LogitsKlArgs&, cudaStream_t);
extern template cudaError_t lk_run<KD_F32>(int, const LogitsKlArgs&, cudaStream_t);

bool logits_kl_fits(int64_t V, int K, int dtype) { return lk_smem(V, K, dtype, 1) <= LK_MAX_SMEM; }

cudaError_t launch_logits_kl(int mode, const void* z, int dtype, int64_t N, int64_t V, int64_t ld, const int32_t* ids,
                             const float* tlog, int K, const float* t_lse, const uint8_t* mask, float tau,
                             float* stats, float* kl, const float* grad_loss, const int32_t* n_valid, void* dz,
                             int64_t ld_dz, uint32_t* err, cudaStream_t s) {
  LogitsKlArgs a{};
  a.z = z; a.dz = dz; a.N = N; a.ld = ld; a.ld_dz = ld_dz; a.V = int(V); a.K = K; a.ids = ids; a.tlog = tlog;
  a.t_lse = t_lse; a.mask = mask; a.tau = tau; a.inv_tau = inverse_tau(tau); a.k = log2e_over_tau(tau);
  a.stats = reinterpret_cast<float4*>(stats); a.kl = kl; a.grad_loss = grad_loss; a.n_valid = n_valid; a.err = err;
  cudaError_t e;
  prof_before(mode == 1 ? "kd_logits_kl_fwd" : mode == 2 ? "kd_logits_kl_bwd" : "kd_logits_kl_step", s);
  KD_DISPATCH_TYPE(dtype, e = lk_run<DT>(mode, a, s));
  prof_after(s);
  return e;
}

// --------------------------------------------------------------- the loss ---
// Mean of kl over the valid rows (0 if there are none) and their number, by one block in a fixed
// order, in fp64.
__global__ void __launch_bounds__(1024) kd_masked_mean_kernel(const float* __restrict__ kl,
                                                              const uint8_t* __restrict__ mask, int64_t N,
                                                              float* __restrict__ loss) {
  __shared__ double sums[32];
  __shared__ int counts[32];
  double sum = 0.0;
  int n = 0;
  for (int64_t i = threadIdx.x; i < N; i += 1024)
    if (mask == nullptr || mask[i] != 0) {
      sum += double(kl[i]);
      ++n;
    }
  const int lane = int(threadIdx.x & 31), warp = int(threadIdx.x >> 5);
  auto reduce = [&] {
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_down_sync(0xffffffffu, sum, o);
    n = __reduce_add_sync(0xffffffffu, n);
  };
  reduce();
  if (lane == 0) {
    sums[warp] = sum;
    counts[warp] = n;
  }
  __syncthreads();
  if (warp == 0) {
    sum = sums[lane];
    n = counts[lane];
    reduce();
    if (lane == 0) *loss = n > 0 ? float(sum / double(n)) : 0.f;
  }
}

cudaError_t launch_masked_mean(const float* kl, const uint8_t* mask, int64_t N, float* loss, cudaStream_t s) {
  prof_before("kd_masked_mean", s);
  kd_masked_mean_kernel<<<1, 1024, 0, s>>>(kl, mask, N, loss);
  prof_after(s);
  return cudaGetLastError();
}

}  // namespace kd
