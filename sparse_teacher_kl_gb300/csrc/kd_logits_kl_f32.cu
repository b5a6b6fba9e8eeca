#include "kd_logits_kl.cuh"

namespace kd {
template cudaError_t lk_run<KD_F32>(int, const LogitsKlArgs&, cudaStream_t);
}  // namespace kd
