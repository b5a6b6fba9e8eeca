// Internal declarations shared by the translation units of libkdkl.so.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/kdkl.h"
#include "kd_host_state.h"

namespace kd {

// Device error word codes (first word of every workspace; the second word
// holds a detail, the third a launch tag).
constexpr uint32_t KD_DEVERR_NONE = 0;
constexpr uint32_t KD_DEVERR_TIMEOUT = 1;
constexpr uint32_t KD_DEVERR_BAD_ID = 2;
constexpr uint32_t KD_DEVERR_BOUNDS = 3;  // KD_DEBUG builds: a computed index out of range (skipped)
constexpr uint32_t KD_DEVERR_NOT_KEPT = 4;  // a backward pass from what no forward pass has kept for it

// Upper bound on any single wait inside a kernel.  A healthy wait lasts
// microseconds; this only stops a kernel that would otherwise hang.
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s

// Workspace control block at offset 0 of every workspace.
struct Ctrl {
  uint32_t err;        // KD_DEVERR_*
  uint32_t err_detail;
  uint32_t topk_reselected;  // top-K: rows selected a second time after a speculative start
  uint32_t pad0;
  int32_t n_valid;     // number of valid positions of the current call
  uint32_t kept;       // cross entropy: what a forward pass has kept here (ce_tag), 0 once it is spent
  uint32_t pad1[58];
};
static_assert(sizeof(Ctrl) == 256, "control block is 256 bytes");

// GEMM engine geometry: one CTA computes a 128 x 256 fp32 tile in tensor
// memory, K staged 64 bf16 (128 B, one swizzle row) at a time.
constexpr int BM = 128;
constexpr int BN = 256;
constexpr int BK = 64;
constexpr int STAGES = 4;
constexpr int STAGE_A_BYTES = BM * BK * 2;  // 16 KB
constexpr int STAGE_B_BYTES = BN * BK * 2;  // 32 KB
constexpr int STAGE_BYTES = STAGE_A_BYTES + STAGE_B_BYTES;
constexpr int GEMM_THREADS = 192;           // TMA warp, MMA warp, 4 epilogue warps
constexpr int STAGING_BYTES = 4 * 2 * 4096; // per epilogue warp: two 32 x 128 B output boxes
constexpr int TMEM_COLS = 512;              // two 256-column fp32 accumulators

// Epilogue kinds of the GEMM engine.
enum EpiKind : int {
  EPI_LSE = 0,    // forward: online logsumexp + teacher-id gather -> partials
  EPI_DZ = 1,     // backward: dZ = scale * (softmax - p) -> bf16 [rows, ldz]
  EPI_STORE = 2,  // C = acc -> fp32 or bf16
  EPI_ACCUM = 3,  // C += acc (fp32)
  EPI_LSE_Z = 4,  // forward-chunked: EPI_LSE plus the raw logits z -> bf16, blocked [V/64][N][64]
  EPI_LSE_H = 5,  // log probabilities: online logsumexp and entropy sum, the token's logit -> partials
  EPI_DZ_LP = 6,  // their gradient: dZ = p (c0 + c1 log2 p) + [v = token] g / tau -> bf16, blocked
  EPI_CE = 7,     // cross entropy: a tile's (max, sum, label's logit, sum of logits) -> partials; with ce_q the
                  // logits in 16 bits (CeCode), blocked as dZ.  EPI_CE + code: without a cap
  EPI_CE_EDGE = 8,   // caps up to CE_CAP_EDGE
  EPI_CE_SPLIT = 9,  // wider ones
};
__host__ __device__ constexpr bool is_ce(int epi) { return epi >= EPI_CE && epi <= EPI_CE_SPLIT; }

// 64-deep k-blocks per ring stage of a CTA-pair launch: two when both operands are
// K-major (the loss sweeps and the teacher projection: each stage one depth-2 box per
// operand), one otherwise (the gradient products, MN-major operands: more, shallower
// stages measured faster there).  The tensor maps of a pair launch are sized for this.
constexpr int pair_kblocks(int a_mn, int b_mn) { return (a_mn == 0 && b_mn == 0) ? 2 : 1; }

struct GemmProblem {
  int M, N, K;           // logical GEMM sizes
  int a_mn, b_mn;        // operand major-ness (0 = K-major)
  int epi;               // EpiKind
  // tile schedule: tiles are (m_blk, n_blk); n_group consecutive n tiles form
  // one unit processed by one CTA in order (used by EPI_LSE).
  int m_tiles, n_tiles, n_group, n_units;
  // split-K (EPI_STORE): the K range is cut into k_splits nearly equal parts; the
  // partial of split s goes to C + s * split_stride (elements).
  int k_splits;
  int64_t split_stride;
  // blocked dZ: operand A (a_blocked) or the EPI_DZ output is the 3-D blocked layout
  // dZ[vocab / 64][row][vocab % 64] (see make_tmap_dz_blocked), so that every TMA box
  // of it is one contiguous run of memory.
  int a_blocked;
  // a_box2 / b_box2 (CTA pairs, MN-major operand): the operand's two 64-column blocks of
  // a stage come in one TMA box of depth 2 from a 3-D map (64, k, blocks), 8 KB apart in
  // shared memory as the MMA reads them; 0: two boxes from a 2-D (or depth-1) map.
  int a_box2, b_box2;
  // a_k3d / b_k3d (CTA pairs with two k-blocks per stage, K-major operand): both come in
  // one box of depth 2 from a 3-D view (64, rows, K / 64); 0: one box per k-block.
  int a_k3d, b_k3d;
  int z_row0;                 // EPI_LSE_Z: row of the stored logits that chunk row 0 maps to
  // cluster: CTAs per cluster, 2 for CTA pairs (cta_pair = 1), else 1.  The CTAs of a
  // pair take consecutive m tiles of the same n tile; n_units counts pairs' units.
  int cluster;
  // cta_pair = 1 (cluster = 2): each pair computes one 256 x 256 tile with tcgen05
  // cta_group::2 MMAs (A split by rows, B by columns between the two CTAs, each CTA
  // loading its own halves; K-major B map box 64 x 128).
  int cta_pair;
  // EPI_STORE / EPI_ACCUM
  void* C;
  int64_t ldc;
  int c_bf16;
  // c_tma = 1 (EPI_STORE, bf16 C, k_splits = 1): the epilogue writes 32 x 64 boxes staged
  // in shared memory with TMA stores through tmap_c (row-major C, box 64 x 32, 128-byte
  // swizzle), clipped at the matrix edges; 0: direct 16-byte stores.
  int c_tma;
  // tile_max (c_tma = 1 only; NULL: none): per row of C and per BN-column tile, the largest
  // bf16-rounded value of the row inside the tile (columns < N; bf16 bits, -inf for a tile
  // of NaNs), at tile_max[row * ld_tile_max + tile] for rows < M.
  uint16_t* tile_max;
  int64_t ld_tile_max;
  // tile_sum (with tile_max; NULL: none): per row and BN-column tile, the sum of
  // 2^((z - m) log2 e) over the row's bf16-rounded values z in the tile (columns < N), m
  // the tile's maximum above (NaN if one of them is NaN), at tile_sum[row * ld_tile_max +
  // tile] for rows < M: with tile_max, the row's logsumexp in pieces.
  float* tile_sum;
  // m_fast = 1 (EPI_STORE / EPI_ACCUM with k_splits = 1): units walk m fastest, so the CTAs
  // in flight share one B tile while the A operand stays in L2 (for a small A and a B
  // larger than L2, as in the teacher projection); 0: n fastest (they share one A slab).
  int m_fast;
  // EPI_LSE / EPI_DZ (rows = tokens of the chunk, cols = vocabulary)
  const int32_t* ids_sorted;  // [rows, K] ascending
  const float* p_sorted;      // [rows, K] teacher probabilities matching ids_sorted
  int Kt;                     // teacher K
  float inv_tau;
  float k;                    // EPI_LSE_H / EPI_DZ_LP: log2(e) / tau
  float4* partials;           // EPI_LSE: [n_units_per_row, rows] (m2, s, G, 0); EPI_LSE_H: (m, s, z_token, u)
  // EPI_LSE_H / EPI_DZ_LP (chunk-relative): the given token of each row; the gradients that
  // reach its log probability and (NULL: none) the entropy
  const int32_t* tokens;
  const float* g_logp;
  const float* g_entropy;
  const float* entropy;
  const float2* row_stats;    // EPI_DZ_LP: [rows] (m, log2 s - (m k - O(m))), in the place of lse; or null
  const float* lse;           // EPI_DZ: [rows] natural-log lse (chunk-relative pointer)
  const uint8_t* mask;        // EPI_DZ: [rows] or null (chunk-relative pointer)
  const float* grad_loss;     // EPI_DZ: device scalar
  const int32_t* n_valid;     // EPI_DZ: device scalar
  uint16_t* dz;               // EPI_DZ: bf16 [rows, ldz]
  int64_t ldz;
  int rows;                   // valid rows of A (tokens in this chunk) for LSE/DZ
  // rows_dev (NULL: none): only the first clamp(*rows_dev - row_first, 0, rows) rows of the chunk
  // exist: the M extent of a product whose A is K-major, the K extent of one whose A is MN-major
  // (there an EPI_STORE takes one k-block of zeros when none exists).
  const int32_t* rows_dev;
  int row_first;
  const int32_t* row_map;     // EPI_STORE without c_tma and splits (NULL: none): row of C that row i goes to, below
  int64_t map_rows;           // map_rows
  const float* alpha;         // EPI_STORE / EPI_ACCUM (NULL: 1): device scalar, a factor of the product
  // EPI_CE: tokens as above; logits capped to ce_cap tanh(z / ce_cap) (0: not); ce_sum: the sum of
  // logits is wanted; ce_q: the 16-bit logits go out through tmap_c
  float ce_cap;
  int ce_sum, ce_q;
  uint32_t* err;
};

// EPI_CE's partials and 16-bit logits belong to CE_COLS columns (half a tile).  What the 16 bits hold depends on the
// softcap c, since dZ takes the cap's slope 1 - (z'/c)^2 from them as well as the probability:
//   CE_CODE_DIST   no cap: the distance from the largest of those columns in steps of 1 / CE_STEPS, 65535 for
//                  anything 32 and further below (e^-32 of the largest, 1.3e-14).  Half a step makes 2.4e-4 of a
//                  probability, an eighth of the rounding of bf16 dZ; bf16 logits would make 2^-8 of every unit of |z|.
//   CE_CODE_EDGE   c up to CE_CAP_EDGE: the sign of z' and w = sqrt(1 - |z'| / c) in steps of 1 / CE_EDGE_STEPS, so
//                  z' = +-c (1 - w^2) and the slope w^2 (2 - w^2).  Half a step is at most 3.1e-5 c of z' (4.9e-4
//                  of a probability at c = 16, 2.4e-4 at 8), and of the slope 6.2e-5 or 3.1e-5 / w of itself, so that
//                  logits near the cap keep theirs: 0.04 % of a slope of 0.01, 0.4 % of 1e-4, 0 at the cap.
//   CE_CODE_SPLIT  wider caps: the distance as above where it is below CE_SPLIT, and beyond, where the probability is
//                  below e^-28 of the largest (7e-13; it is taken as at most that) and only the slope counts,
//                  w = sqrt((z' + c) / 2 c) in steps of 1 / CE_FAR_STEPS, the slope 4 w^2 (1 - w^2).  A distance's half
//                  step is 2.4e-4 / c of z' / c: 3e-5 of a slope at c = 16.
constexpr int CE_COLS = BN / 2;
constexpr int CE_CHUNK_K = 512;   // depth of EPI_CE's partial sums
constexpr float CE_STEPS = 2048.f;
enum CeCode : int { CE_CODE_DIST = 0, CE_CODE_EDGE = 1, CE_CODE_SPLIT = 2 };
constexpr float CE_CAP_EDGE = 16.f;
constexpr float CE_EDGE_STEPS = 32767.f;
constexpr float CE_SPLIT = 28.f;
constexpr uint32_t CE_SPLIT_CODE = uint32_t(CE_SPLIT * CE_STEPS);
constexpr float CE_FAR_STEPS = float(65535 - CE_SPLIT_CODE);
__host__ __device__ inline CeCode ce_code(float cap) {
  return !(cap > 0.f) ? CE_CODE_DIST : cap <= CE_CAP_EDGE ? CE_CODE_EDGE : CE_CODE_SPLIT;
}

// Host helpers of the C ABI.
inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline kd_status map_cuda(cudaError_t e) { return e == cudaSuccess ? KD_OK : KD_ERR_CUDA; }
// 1 / tau and log2(e) / tau of the calls on dense logits and of the scores from hidden states, finite
// for every tau > 0: below 3e-39 (4e-39) they would be infinite, and 0 times them NaN.
inline float inverse_tau(float tau) { return 1.0f / tau <= FLT_MAX ? 1.0f / tau : FLT_MAX; }
inline float log2e_over_tau(float tau) {
  const double k = 1.4426950408889634 / double(tau);
  return k <= double(FLT_MAX) ? float(k) : FLT_MAX;
}
// Rows, columns and depths are counted in 32 bits, up to a tile (or a block's step) behind the last one.
constexpr int64_t KD_MAX_EXTENT = 0x7fffffffLL - 1023;
// What every call on hidden states and a head checks: sizes, chunk, alignment, temperature.
kd_status check_proj_args(const void* H, const void* W, int64_t N, int64_t d, int64_t V, int64_t chunk, float tau);
// KD_OK if the current device is an sm_103 GPU.
kd_status check_device();

// Tensor maps (kd_abi.cu).
bool make_tmap_2d_bf16(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer,
                       uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_outer);
// dZ chunk in blocked layout: [nvb = ceil(V/64)][rows_pad][64] bf16; dims {64, rows, nvb},
// box {64, box_rows, 1}, 128-byte swizzle.
bool make_tmap_dz_blocked(CUtensorMap* map, const void* base, uint64_t rows, uint64_t rows_pad, uint64_t nvb,
                          uint32_t box_rows, uint32_t box_depth = 1);
// 3-D view (64, rows, cols / 64) of a row-major bf16 matrix whose column count is a
// multiple of 64, box (64, box_rows, 2): two 64-column blocks per TMA box (two k-blocks
// of a K-major operand, or two column blocks of an MN-major one).
bool make_tmap_mn2_bf16(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint64_t row_stride_bytes,
                        uint32_t box_rows);
bool make_tmap_2d_u8(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer, uint64_t row_stride_bytes,
                     uint32_t box_inner, uint32_t box_outer);
bool make_tmap_2d_f32(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer,
                      uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_outer);

// Raise a kernel's dynamic shared-memory limit to `bytes` once per device (safe from
// several host threads; `done` is the kernel's own per-device record).
inline cudaError_t smem_attr_once(PerDevice<int>& done, const void* func, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int v = 0;
  const int rc = done.get(dev, &v, [&](int, int* out) {
    *out = 1;
    return int(cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
  });
  return rc == 0 ? cudaSuccess : (rc > 0 ? cudaError_t(rc) : cudaErrorInvalidDevice);
}

// Launchers (return a cudaError_t).
// tc: output map for the epilogues that write through TMA (EPI_ACCUM: fp32 C,
// box 32 x 32; EPI_DZ: bf16 dZ, box 64 x 32; both 128-byte swizzle); ignored
// by the others.
void set_cluster(GemmProblem& p);
cudaError_t launch_gemm(const GemmProblem& p, const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc,
                        int grid, cudaStream_t s);
int gemm_max_grid();

// Top-K of every row of X [N, ld] bf16 (columns [0, V)): ids and values [N, K], optionally
// the row logsumexp lse [N] and the dropped teacher mass dropped [N] (NULL: not wanted).
// err: the workspace control block's error word (its third word counts rows that a
// speculative start made select twice).  scratch: topk_scratch_bytes(N, K) bytes, 256-byte
// aligned.  tile_max (NULL: none): per row, the maxima of ntiles disjoint column ranges of
// the row (bf16 bits, [N, ld_tile_max]); with ntiles >= K their K-th largest is a lower
// bound of the row's K-th largest value and starts the row.  lse_known (NULL: none; only
// where topk_takes_known_lse(K)): the rows' logsumexp, already computed, for the dropped
// mass; the selection then computes none (lse must be NULL).
size_t topk_scratch_bytes(int64_t N, int K);
bool topk_takes_known_lse(int K);
cudaError_t launch_topk(const uint16_t* X, int64_t N, int64_t V, int64_t ld, int K, int32_t* ids,
                        float* vals, float* lse, float* dropped, uint32_t* err, void* scratch, cudaStream_t s,
                        const uint16_t* tile_max = nullptr, int64_t ld_tile_max = 0, int ntiles = 0,
                        const float* lse_known = nullptr);
// Row logsumexp [rows] from the per-tile maxima and sums of a projection's epilogue
// (GemmProblem::tile_max, tile_sum; ntiles of them per row, row stride ld).
cudaError_t launch_tile_lse(const uint16_t* tile_max, const float* tile_sum, int64_t ld, int ntiles, int64_t rows,
                            float* lse, cudaStream_t s);

cudaError_t launch_count_valid(const uint8_t* mask, int64_t N, int32_t* n_valid, cudaStream_t s);
cudaError_t launch_teacher_prologue(const int32_t* ids, const float* tlog, int rows, int K, int64_t V,
                                    float inv_tau, int32_t* ids_sorted, float* p_sorted, float* negent,
                                    uint32_t* err, int64_t row0, cudaStream_t s);
cudaError_t launch_lse_combine(const float4* partials, int n_units_per_row, int rows, const float* negent,
                               float inv_tau, float* lse_out, float* kl_out, cudaStream_t s);
// Log probability, logsumexp and entropy (NULL: not wanted) of each row from EPI_LSE_H's partials.
cudaError_t launch_logprob_combine(const float4* partials, int n_units_per_row, int rows, int64_t V,
                                   const int32_t* tokens, const uint8_t* mask, float tau, float* logp, float* lse,
                                   float* entropy, uint32_t* err, int64_t row0, cudaStream_t s);
// GemmProblem::row_stats of each row from EPI_LSE_H's partials.
cudaError_t launch_logprob_row_stats(const float4* partials, int n_units_per_row, int rows, float tau, float2* row_stats,
                                     cudaStream_t s);
// EPI_LSE_H's partials for up to FEW_ROWS rows without the tensor cores; *units: how many per row
// were written (at most max_units).  Faster than the engine's 128-row tiles for one row where W has
// to come from HBM, and for two where that takes longer than their logits' sums: where W has more
// than FEW_ROW_BYTES for each row, and the vocabulary a unit (BN tokens, as many as the partials have
// room for) for every SM.  us, this / the engine, for a V x d head:
//              4096x256 50257x768 50257x1600 201088x512 151936x1024 50257x4096 151936x2048 201088x2880
//   W in MB       2        77        161        206        311         412        622        1158
//   one row     18/13     29/26      45/49      52/62      60/80      78/103     102/147    190/230
//   two         25/13     37/27      54/51      69/62      74/84      90/102     113/148    209/229
// and with too few units: 32000 x 4096 66/69 and 76/68, 32000 x 8192 117/110 and 130/110, 10000 x 8192
// 105/65 and 118/64; three rows at 1158 MB 298/224, four 298/227.
constexpr int FEW_ROWS = 2;
constexpr int64_t FEW_ROW_BYTES = 150000000;
constexpr int FEW_MAX_SMEM = 200 * 1024;  // the hidden states in fp32: a limit on rows * d
cudaError_t launch_logprob_few(const uint16_t* H, const uint16_t* W, int rows, int d, int64_t V, const int32_t* tokens,
                               const uint8_t* mask, float tau, float4* partials, int max_units, int* units,
                               cudaStream_t s);
cudaError_t launch_loss_reduce(const float* kl, const uint8_t* mask, int64_t N, const int32_t* n_valid,
                               float* loss_out, cudaStream_t s);

cudaError_t launch_wait_timeout(uint32_t* err, uint64_t limit_ns, cudaStream_t s);
cudaError_t launch_dz_from_z(const uint16_t* z, int64_t N, int64_t c0, int rows, int64_t V, int64_t nvb,
                             int64_t rows_pad, const float* lse, const uint8_t* mask, const float* grad_loss,
                             const int32_t* n_valid, float inv_tau, const int32_t* ids_sorted, const float* p_sorted,
                             int K, uint16_t* dz, cudaStream_t s);
cudaError_t launch_split_reduce(const float* parts, int splits, int64_t split_stride, int64_t count, void* out,
                                int out_bf16, cudaStream_t s);

// Dense logits [N, ld] of element type `dtype` (kd_dtype), see kdkl.h.
cudaError_t launch_logprobs_fwd(const void* z, int dtype, int64_t N, int64_t V, int64_t ld, const int32_t* tokens,
                                int M, const uint8_t* mask, float tau, int top, float* logp, float* lse,
                                float* entropy, int32_t* top_ids, float* top_logp, uint32_t* err, cudaStream_t s);
cudaError_t launch_logprobs_bwd(const void* z, int dtype, int64_t N, int64_t V, int64_t ld, const int32_t* tokens,
                                int M, const uint8_t* mask, float tau, const float* lse, const float* entropy,
                                const float* g_logp, const float* g_ent, void* dz, int64_t ld_dz, uint32_t* err,
                                cudaStream_t s);
// mode: 1 = forward (stats, kl), 2 = backward (stats -> dz), 3 = both in one pass (kl, dz).
bool logits_kl_fits(int64_t V, int K, int dtype);
cudaError_t launch_logits_kl(int mode, const void* z, int dtype, int64_t N, int64_t V, int64_t ld, const int32_t* ids,
                             const float* tlog, int K, const float* t_lse, const uint8_t* mask, float tau,
                             float* stats, float* kl, const float* grad_loss, const int32_t* n_valid, void* dz,
                             int64_t ld_dz, uint32_t* err, cudaStream_t s);

// loss = mean of kl over the valid rows, 0 if there are none.
cudaError_t launch_masked_mean(const float* kl, const uint8_t* mask, int64_t N, float* loss, cudaStream_t s);

// 8-bit integers (kd_int8.cu).  ws: gemm_int8_scratch bytes, its first 256 left alone; aligned_rows: the rows of
// B start on 16-byte boundaries.
// Rows that do not are copied (to rows of Kw, a multiple of 16) where gemm_int8_copies_rows says so.
bool gemm_int8_copies_rows(int64_t M, int64_t N, int64_t K);
cudaError_t launch_int8_rows(const int8_t* B, int64_t ldb, int64_t N, int64_t K, int64_t Kw, void* out,
                             cudaStream_t s);
size_t gemm_int8_scratch(int64_t M, int64_t N, int64_t K, bool aligned_rows);
cudaError_t launch_gemm_int8(const int8_t* A, int64_t lda, const float* a_scale, const int8_t* B, int64_t ldb,
                             const float* b_scale, void* C, int dtype, int64_t ldc, int64_t M, int64_t N, int64_t K,
                             uint8_t* ws, uint32_t* err, cudaStream_t s);
cudaError_t launch_quantize_int8(const void* x, int dtype, int64_t N, int64_t d, int64_t ld, int8_t* q, int64_t ldq,
                                 float* scale, cudaStream_t s);

constexpr int KD_MAX_SPLITS = 8;

// Device address of the library's own scratch array (kd_fused_kl_fwd_static) on the
// current device, looked up once per device and context.
kd_status static_scratch_address(void** out);

// Profiling hooks (kd_abi.cu): bracket a launch with events when enabled.
void prof_before(const char* name, cudaStream_t s);
void prof_after(cudaStream_t s);

}  // namespace kd
