// The C ABI of the 8-bit calls (declared in include/kdkl.h): argument checks, workspace layout and the chunk
// loop of the quantised teacher.  Host code only.
#include "kd_internal.h"

using namespace kd;

namespace {

constexpr int64_t kMaxInt = 0x7fffffffLL;

size_t out_size(int dtype) { return dtype == KD_F32 ? 4 : 2; }
bool rows16(const void* B, int64_t ldb) { return aligned(B, 16) && ldb % 16 == 0; }
bool ok4(const void* p) { return p != nullptr && aligned(p, 4); }

// An integer matrix [rows, K] with row stride ld and its scales.
bool ok_matrix(const void* q, int64_t ld, const void* scale, int64_t rows, int64_t K) {
  return q && rows >= 1 && rows <= KD_MAX_EXTENT && K >= 1 && K <= KD_MAX_INT8_K && ld >= K && ok4(scale);
}

struct TopkLayout {
  size_t logits, gemm, weights, scratch, total;
  int64_t ldz, ldw;  // ldw: row stride of the copied weights, 0 where they are read in place
};

TopkLayout topk_layout(int64_t N, int64_t dt, int64_t V, int K, int64_t chunk, bool aligned_rows) {
  TopkLayout L{};
  const int64_t c = chunk < N ? chunk : N;
  L.ldz = (V + 7) / 8 * 8;
  L.logits = sizeof(Ctrl);
  // weights whose rows do not start on 16-byte boundaries: copied once for all chunks
  L.ldw = !aligned_rows && gemm_int8_copies_rows(c, V, dt) ? (dt + 15) / 16 * 16 : 0;
  L.gemm = align_up(L.logits + size_t(c) * size_t(L.ldz) * 2, 256);
  // the last chunk is shorter, and may take the other way
  const int64_t last = (N - 1) % c + 1;
  const bool in_place = aligned_rows || L.ldw;
  const size_t one = gemm_int8_scratch(c, V, dt, in_place), two = gemm_int8_scratch(last, V, dt, in_place);
  L.weights = align_up(L.gemm + (one > two ? one : two), 256);
  L.scratch = align_up(L.weights + size_t(V) * size_t(L.ldw), 256);
  L.total = L.scratch + align_up(topk_scratch_bytes(c, K), 256);
  return L;
}

}  // namespace

extern "C" {

int kd_quantize_int8(const void* x, int dtype, int64_t N, int64_t d, int64_t ld, int8_t* q_out, int64_t ld_q,
                     float* scale_out, void* stream) {
  if (N < 1 || N > kMaxInt || d < 1 || d > KD_MAX_EXTENT || ld < d || ld_q < d) return KD_ERR_INVALID_ARG;
  if (dtype != KD_BF16 && dtype != KD_F16 && dtype != KD_F32) return KD_ERR_INVALID_ARG;
  if (!x || !aligned(x, out_size(dtype)) || !q_out || !ok4(scale_out)) return KD_ERR_INVALID_ARG;
  kd_status st = check_device();
  if (st != KD_OK) return st;
  return map_cuda(launch_quantize_int8(x, dtype, N, d, ld, q_out, ld_q, scale_out, static_cast<cudaStream_t>(stream)));
}

size_t kd_gemm_int8_workspace(int64_t M, int64_t N, int64_t K, int b_rows_aligned) {
  if (M < 1 || N < 1 || K < 1) return 0;
  return gemm_int8_scratch(M, N, K, b_rows_aligned != 0);
}

int kd_gemm_int8(const int8_t* A, int64_t lda, const float* a_scale, const int8_t* B, int64_t ldb, const float* b_scale,
                 void* C, int dtype, int64_t ldc, int64_t M, int64_t N, int64_t K, void* ws, size_t ws_bytes,
                 void* control, void* stream) {
  if (!ok_matrix(A, lda, a_scale, M, K) || !ok_matrix(B, ldb, b_scale, N, K)) return KD_ERR_INVALID_ARG;
  if (dtype != KD_BF16 && dtype != KD_F16 && dtype != KD_F32) return KD_ERR_INVALID_ARG;
  if (!C || !aligned(C, out_size(dtype)) || ldc < N) return KD_ERR_INVALID_ARG;
  if (((N + 127) / 128) * ((M + 127) / 128) > kMaxInt) return KD_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 256) || ws_bytes < gemm_int8_scratch(M, N, K, rows16(B, ldb)) || !control ||
      !aligned(control, 256))
    return KD_ERR_WORKSPACE;
  kd_status st = check_device();
  if (st != KD_OK) return st;
  return map_cuda(launch_gemm_int8(A, lda, a_scale, B, ldb, b_scale, C, dtype, ldc, M, N, K, static_cast<uint8_t*>(ws),
                                   &static_cast<Ctrl*>(control)->err, static_cast<cudaStream_t>(stream)));
}

size_t kd_teacher_topk_int8_workspace(int64_t N, int64_t dt, int64_t V, int K, int64_t chunk, int w_rows_aligned) {
  if (N < 1 || dt < 1 || V < 1 || K < 1 || chunk < 1) return 0;
  return topk_layout(N, dt, V, K, chunk, w_rows_aligned != 0).total;
}

int kd_teacher_topk_int8(const int8_t* Ht, int64_t ld_h, const float* h_scale, const int8_t* Wt, int64_t ld_w,
                         const float* w_scale, int64_t N, int64_t dt, int64_t V, int K, int64_t chunk,
                         int32_t* ids_out, float* vals_out, float* lse_out, float* dropped_out, void* ws,
                         size_t ws_bytes, void* control, void* stream) {
  if (!ok_matrix(Ht, ld_h, h_scale, N, dt) || !ok_matrix(Wt, ld_w, w_scale, V, dt)) return KD_ERR_INVALID_ARG;
  if (K < 1 || K > KD_MAX_K || int64_t(K) > V || chunk < 1) return KD_ERR_INVALID_ARG;
  if (!ok4(ids_out) || !ok4(vals_out) || !aligned(lse_out, 4) || !aligned(dropped_out, 4)) return KD_ERR_INVALID_ARG;
  const TopkLayout L = topk_layout(N, dt, V, K, chunk, rows16(Wt, ld_w));
  if (!ws || !aligned(ws, 256) || ws_bytes < L.total || !control || !aligned(control, 256)) return KD_ERR_WORKSPACE;
  kd_status st = check_device();
  if (st != KD_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* w8 = static_cast<uint8_t*>(ws);
  uint16_t* logits = reinterpret_cast<uint16_t*>(w8 + L.logits);
  uint32_t* err = &static_cast<Ctrl*>(control)->err;
  if (L.ldw) {
    if (launch_int8_rows(Wt, ld_w, V, dt, L.ldw, w8 + L.weights, s) != cudaSuccess) return KD_ERR_CUDA;
    Wt = reinterpret_cast<const int8_t*>(w8 + L.weights);
    ld_w = L.ldw;
  }
  for (int64_t c0 = 0; c0 < N; c0 += chunk) {
    const int64_t n = (N - c0) < chunk ? (N - c0) : chunk;
    // the chunk's logits, rounded once to bf16, then their exact top-K
    cudaError_t e = launch_gemm_int8(Ht + c0 * ld_h, ld_h, h_scale + c0, Wt, ld_w, w_scale, logits, KD_BF16, L.ldz, n, V,
                                     dt, w8 + L.gemm, err, s);
    if (e == cudaSuccess)
      e = launch_topk(logits, n, V, L.ldz, K, ids_out + c0 * K, vals_out + c0 * K, lse_out ? lse_out + c0 : nullptr,
                      dropped_out ? dropped_out + c0 : nullptr, err, w8 + L.scratch, s);
    if (e != cudaSuccess) return KD_ERR_CUDA;
  }
  return KD_OK;
}

}  // extern "C"
