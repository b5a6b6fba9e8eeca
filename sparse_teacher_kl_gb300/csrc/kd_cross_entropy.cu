// Softmax cross entropy from hidden states: the row-wise steps around the projection engine, and the
// host side of kd_fused_cross_entropy_*.  With z' = z, or c tanh(z / c) for a softcap c, over the V
// logits z = h W^T of a position with label y,
//   lse    = logsumexp(z')
//   loss_n = lse - (1 - e) z'_y - (e / V) sum_v z'_v + l lse^2       (e label smoothing, l z-loss)
//   loss   = sum_n loss_n / n_valid
//   dZ_v   = G ((1 + 2 l lse) p_v - e / V - (1 - e) [v = y]) (1 - (z'_v / c)^2),   G = grad / n_valid
//   grad_H = dZ W,   grad_W = dZ^T H
//
// What a step cannot do without is 6 N d V operations (one projection, two gradient products); what it
// must move is H, W and the two gradients.  The usual way to keep no logits is to project twice (8 N d V).
// Here the projection's epilogue leaves each chunk's logits in 16 bits (CeCode: distances from the largest of
// their CE_COLS columns, with a softcap a code that keeps its slope; in the buffer that dZ needs anyway), and once a row's sum is
// known one pass over that buffer turns them into bf16 dZ where they lie: 6 bytes moved for each logit
// against 2 d operations, 0.9 ns against 3.3 ns per thousand at d = 2880.  The label's own entry, where
// p_y - 1 would cancel, comes from its fp32 logit.
//
// Positions without a loss (mask 0, or the ignored label) cost nothing: the others are gathered to the
// front, in order, and the products stop after the last of them (GemmProblem::rows_dev).  Their hidden states
// are never read, so they may hold anything.
//
// Measured (one pass of a step, H and W bf16): 4096 x 2880 x 201088 9.3 ms, of it the projection 2.6, dZ 0.53 (6.2 TB/s),
// the products 2.7 each (1.75 PFLOP/s); 8192 x 2048 x 32000 with 5 % of the labels ignored 2.1 ms (fused_logprobs with
// its gradient, which projects twice: 2.7); 4096 x 4096 x 151936 with 65 % ignored 3.65 ms, none ignored 9.0.  A softcap
// adds 2 to 3 % to a step: 4096 x 2048 x 128000 4.05 ms, with c = 8 4.15, with 30 4.2.  kd_ce_combine_kernel's
// loops over the phases are unrolled whole and spill 600 bytes a thread (8 to 45 us of a step).
#include <math.h>
#include <string.h>

#include <initializer_list>
#include <type_traits>

#include "kd_device.cuh"
#include "kd_internal.h"

namespace kd {

namespace {

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kMinSoftcap = 1e-6f;  // its square and reciprocal are ordinary numbers

__device__ __forceinline__ bool has_loss(const int32_t* labels, const uint8_t* mask, int64_t i, int ignore) {
  return labels[i] != ignore && (mask == nullptr || mask[i] != 0);
}

// ------------------------------------------------------------------ positions ---
// list[0 .. n_valid): the positions that have a loss, ascending.  The others' outputs are set to 0.  One block,
// eight positions a thread and sweep, so that each sweep's loads are in flight together.
constexpr int LIST_THREADS = 1024, LIST_EACH = 8;

__global__ void __launch_bounds__(LIST_THREADS)
    kd_ce_list_kernel(const int32_t* __restrict__ labels, const uint8_t* __restrict__ mask, int64_t N, int ignore,
                      int32_t* __restrict__ list, int32_t* __restrict__ n_valid, float* __restrict__ lse,
                      float* __restrict__ losses, uint32_t* __restrict__ kept, uint32_t tag) {
  __shared__ int warp_sum[LIST_THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int base = 0;
  for (int64_t i0 = 0; i0 < N; i0 += int64_t(LIST_THREADS) * LIST_EACH) {
    const int64_t first = i0 + int64_t(threadIdx.x) * LIST_EACH;
    uint32_t on = 0;
#pragma unroll
    for (int j = 0; j < LIST_EACH; ++j)
      if (first + j < N && has_loss(labels, mask, first + j, ignore)) on |= 1u << j;
    const int mine = __popc(on);
    int sum = mine;  // inclusive over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll 8
    for (int w = 0; w < LIST_THREADS / 32; ++w) {
      const int v = warp_sum[w];
      before += w < warp ? v : 0;
      total += v;
    }
    int at = base + before + sum - mine;
#pragma unroll
    for (int j = 0; j < LIST_EACH; ++j) {
      if (first + j >= N) break;
      if (on >> j & 1u) {
        list[at++] = int32_t(first + j);
      } else {
        lse[first + j] = 0.f;
        losses[first + j] = 0.f;
      }
    }
    base += total;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    *n_valid = base;
    *kept = tag;
  }
}

// The start of a backward pass from a kept forward pass: what is not there (another call's, or already spent) leaves
// no valid position, so that nothing of it is used as an index; grad_H zero, for the positions without a loss.
__global__ void __launch_bounds__(256)
    kd_ce_begin_kernel(Ctrl* __restrict__ ctrl, uint32_t tag, uint4* __restrict__ grad_H, int64_t vecs, uint32_t* err) {
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (ctrl->kept != tag) {
      raise_error(err, KD_DEVERR_NOT_KEPT, 0);
      ctrl->n_valid = 0;
    }
    ctrl->kept = 0;
  }
  for (int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; i < vecs; i += int64_t(gridDim.x) * blockDim.x)
    grad_H[i] = make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ int chunk_rows(const int32_t* n_valid, int64_t c0, int cap) {
  const int64_t n = int64_t(*n_valid) - c0;
  return int(n < 0 ? 0 : n > cap ? cap : n);
}

// Rows that the products read: whole 64-row blocks, one at least.
__device__ __forceinline__ int read_rows(int n) { return n < 1 ? 64 : (n + 63) / 64 * 64; }

// A chunk's hidden states and labels to the front; zero rows after the last, as far as the products read.  With
// zero_H (first chunk of a step): the gradients of positions without a loss.  A warp copies a row.
constexpr int GATHER_WARPS = 8;

__global__ void __launch_bounds__(GATHER_WARPS * 32)
    kd_ce_gather_kernel(const uint16_t* __restrict__ H, const int32_t* __restrict__ labels,
                        const uint8_t* __restrict__ mask, int64_t N, int64_t d, int ignore,
                        const int32_t* __restrict__ list, const int32_t* __restrict__ n_valid, int64_t c0, int cap,
                        int rows_pad, uint16_t* __restrict__ Hc, int32_t* __restrict__ labels_c,
                        void* __restrict__ zero_H, int64_t zero_vecs, uint32_t* err) {
  const int lane = threadIdx.x & 31;
  const int64_t w0 = int64_t(blockIdx.x) * GATHER_WARPS + (threadIdx.x >> 5), step = int64_t(gridDim.x) * GATHER_WARPS;
  const int n = chunk_rows(n_valid, c0, cap);
  const int end = min(read_rows(n), rows_pad);
  const int64_t vecs = d / 8;
  for (int64_t r = w0; r < end; r += step) {
    uint4* dst = reinterpret_cast<uint4*>(Hc + r * d);
    const int64_t i = r < n ? list[c0 + r] : 0;
    if (r < n && KD_DCHECK(i >= 0 && i < N, err, 0x2000)) {
      const uint4* src = reinterpret_cast<const uint4*>(H + i * d);
      if (lane == 0) labels_c[r] = labels[i];
#pragma unroll 4
      for (int64_t v = lane; v < vecs; v += 32) dst[v] = __ldg(src + v);
    } else {
      for (int64_t v = lane; v < vecs; v += 32) dst[v] = make_uint4(0, 0, 0, 0);
    }
  }
  if (zero_H == nullptr) return;
  for (int64_t i = w0; i < N; i += step) {
    if (has_loss(labels, mask, i, ignore)) continue;
    uint4* dst = reinterpret_cast<uint4*>(zero_H) + i * zero_vecs;
    for (int64_t v = lane; v < zero_vecs; v += 32) dst[v] = make_uint4(0, 0, 0, 0);
  }
}

// ------------------------------------------------------------------ row sums ---
// A row's tiles put together: its loss and logsumexp to the position's place and, for a step, what dZ
// takes of it: (M, a, b, dz_y) with dZ_v = (a e^(z'_v - M) - b) slope_v, M the largest logit: 1 / S is in a, since
// M + ln S would be rounded at its own size (logits of 1e6: to 1/16).  dZ leaves out alpha = G (1 - e), which is every
// entry's and joins the fp32 products: the label's entry is then 1 - p_y / (1 - e) and not G times that, whose
// rounding to bf16 would be the same in every row that the model has not learnt (p_y near 0), up to 2^-8 of the
// gradients.  32 threads share a row's tiles (as the other combines: a thread's tiles are a chain of dependent
// exponentials).
constexpr int CC_ROWS = 32, CC_PHASES = 32;

struct CeCombine {
  const float4* partials;
  int tiles, rows_pad, cap;
  int64_t c0, N, V;
  const int32_t *list, *n_valid, *labels_c;
  float smooth, z_loss, softcap;
  float *lse, *losses;
  float4* row_stats;
  uint32_t* err;
};

__global__ void __launch_bounds__(CC_ROWS * CC_PHASES) kd_ce_combine_kernel(const CeCombine a) {
  __shared__ float4 sm[CC_PHASES][CC_ROWS];
  const int x = threadIdx.x, y = threadIdx.y;
  const int r = blockIdx.x * CC_ROWS + x;
  const int n = chunk_rows(a.n_valid, a.c0, a.cap);
  if (int(blockIdx.x) * CC_ROWS >= n) return;
  float M = -INFINITY, S = 0.f, Y = 0.f, Z = 0.f;
  if (r < n) {
#pragma unroll 4
    for (int u = y; u < a.tiles; u += CC_PHASES) {
      const float4 q = a.partials[size_t(u) * a.rows_pad + r];
      Y += q.z;
      Z += q.w;
      if (q.x > M) {
        S = fmaf(S, exp2f((M - q.x) * kLog2E), q.y);
        M = q.x;
      } else if (q.x != -INFINITY) {
        S = fmaf(q.y, exp2f((q.x - M) * kLog2E), S);
      } else {
        S += q.y;  // 0, or NaN of a tile that holds one
      }
    }
  }
  sm[y][x] = make_float4(M, S, Y, Z);
  __syncthreads();
  if (y != 0 || r >= n) return;
  for (int k = 1; k < CC_PHASES; ++k) M = fmaxf(M, sm[k][x].x);
  S = Y = Z = 0.f;
  for (int k = 0; k < CC_PHASES; ++k) {
    const float4 q = sm[k][x];
    S += q.x == -INFINITY ? q.y : q.y * exp2f((q.x - M) * kLog2E);
    Y += q.z;
    Z += q.w;
  }
  const int64_t pos = a.list[a.c0 + r];
  if (!KD_DCHECK(pos >= 0 && pos < a.N, a.err, 0x2001)) return;
  const int32_t label = a.labels_c[r];
  const bool bad = label < 0 || int64_t(label) >= a.V;
  if (bad) raise_error(a.err, KD_DEVERR_BAD_ID, uint32_t(pos));
  const float ln_s = logf(S), lse = M + ln_s;
  // as a difference of logits: lse and z_y would each be rounded at their own size
  const float nll = ln_s - (Y - M);
  // (a label at -inf: nll is +inf, and so is the loss, though the mean is at -inf with it)
  const float mean_off = a.smooth > 0.f && Y != -INFINITY ? Y - Z / float(a.V) : 0.f;
  a.lse[pos] = lse;
  a.losses[pos] = bad ? __int_as_float(0x7FC00000) : nll + a.smooth * mean_off + a.z_loss * lse * lse;
  if (a.row_stats == nullptr) return;
  float4 st = make_float4(M, 0.f, 0.f, 0.f);
  if (!bad) {
    const float scale = 1.f / (1.f - a.smooth), of_p = scale * fmaf(2.f * a.z_loss, lse, 1.f);
    st.y = of_p / S;
    st.z = scale * (a.smooth / float(a.V));
    st.w = of_p * exp2f(-nll * kLog2E) - st.z - 1.f;
    if (a.softcap > 0.f) {
      const float e = fmaxf(a.softcap - fabsf(Y), 0.f) / a.softcap;
      st.w *= e * (2.f - e);
    }
  }
  a.row_stats[r] = st;
}

// ------------------------------------------------------------------ dZ ---
// The chunk's 16-bit codes to bf16 dZ, in place ([V / 64][row][64], both).  A block takes 128 rows of
// CE_COLS columns: 8 lanes to a 128-byte row of a 64-column block, 8 vectors of 16 bytes in flight a thread.
// Bound by HBM: 4 bytes a logit.
constexpr int DQ_ROWS = 128, DQ_BLOCKS = CE_COLS / 64;

// What the entries of a row's CE_COLS columns take of it: dZ = (a e^(z' - M) - b) slope.
struct DzRow {
  float a, b, m, M, shift, cap, cap_inv;
};

// An entry from its code (CeCode; FAR as for ce_codes).  Where no column of the CE_COLS is above -inf, m - M is -inf
// and p is 0.
template <CeCode CODE, bool FAR = true>
__device__ __forceinline__ float dz_of(uint32_t q, const DzRow& r) {
  if (CODE == CE_CODE_EDGE) {
    const float w = float(q & 0x7FFFu) * (1.f / CE_EDGE_STEPS), e = w * w;  // e = 1 - |z'| / c
    const float z = __uint_as_float(__float_as_uint(fmaf(-r.cap, e, r.cap)) | (q & 0x8000u) << 16);
    return fmaf(r.a, ex2_approx((z - r.M) * kLog2E), -r.b) * (e * (2.f - e));
  }
  float shift = fmaf(float(q), -kLog2E / CE_STEPS, r.shift);
  if (CODE == CE_CODE_DIST) return fmaf(r.a, ex2_approx(shift), -r.b);
  const float z = fmaf(float(q), -1.f / CE_STEPS, r.m);
  float e = fmaxf(r.cap - fabsf(z), 0.f) * r.cap_inv, slope = e * (2.f - e);
  if (FAR && q >= CE_SPLIT_CODE) {
    const float w = float(q - CE_SPLIT_CODE) * (1.f / CE_FAR_STEPS);
    e = w * w;  // (z' + c) / 2 c, whose step may be wide (c / 4096): the distance is known to be CE_SPLIT at least
    shift = fmaf(fminf(r.cap * fmaf(2.f, e, -1.f) - r.m, -CE_SPLIT), kLog2E, r.shift);
    slope = 4.f * e * (1.f - e);
  }
  return fmaf(r.a, ex2_approx(shift), -r.b) * slope;
}

template <CeCode CODE>
__global__ void __launch_bounds__(256)
    kd_ce_dz_kernel(uint4* __restrict__ dz, int rows_pad, int64_t nvb, const float4* __restrict__ partials, int ld_part,
                    const float4* __restrict__ row_stats, const int32_t* __restrict__ labels_c,
                    const int32_t* __restrict__ n_valid, int64_t c0, int cap, float softcap,
                    const float* __restrict__ grad_loss, float label_weight, float* __restrict__ alpha) {
  const int n = chunk_rows(n_valid, c0, cap);
  const int end = min(read_rows(n), rows_pad);
  if (blockIdx.x == 0 && threadIdx.x == 0)  // the gradients' common factor, see CeCombine
    *alpha = *n_valid > 0 ? (grad_loss ? *grad_loss : 1.f) * label_weight / float(*n_valid) : 0.f;
  const uint32_t row_blocks = uint32_t(cap + DQ_ROWS - 1) / DQ_ROWS;
  const int tile = int(blockIdx.x / row_blocks), lane8 = threadIdx.x & 7;
  const int first = int(blockIdx.x - uint32_t(tile) * row_blocks) * DQ_ROWS, r0 = first + (threadIdx.x >> 3);
  if (first >= end) return;
  const int vb0 = tile * DQ_BLOCKS;
  uint4 v[DQ_ROWS / 32][DQ_BLOCKS];
#pragma unroll
  for (int h = 0; h < DQ_ROWS / 32; ++h)
#pragma unroll
    for (int b = 0; b < DQ_BLOCKS; ++b)
      if (r0 + h * 32 < n && vb0 + b < nvb) v[h][b] = dz[(size_t(vb0 + b) * rows_pad + r0 + h * 32) * 8 + lane8];
#pragma unroll
  for (int h = 0; h < DQ_ROWS / 32; ++h) {
    const int r = r0 + h * 32;
    if (r >= end) return;
    if (r >= n) {
#pragma unroll
      for (int b = 0; b < DQ_BLOCKS; ++b)
        if (vb0 + b < nvb) dz[(size_t(vb0 + b) * rows_pad + r) * 8 + lane8] = make_uint4(0, 0, 0, 0);
      continue;
    }
    const float4 st = row_stats[r];
    DzRow row{};
    row.a = st.y; row.b = st.z; row.M = st.x;
    row.m = partials[size_t(tile) * ld_part + r].x;
    row.shift = (row.m - row.M) * kLog2E;
    if (CODE != CE_CODE_DIST) {
      row.cap = softcap;
      row.cap_inv = 1.f / softcap;
    }
    const int label = labels_c[r];
#pragma unroll
    for (int b = 0; b < DQ_BLOCKS; ++b) {
      if (vb0 + b >= nvb) break;
      const uint32_t w[4] = {v[h][b].x, v[h][b].y, v[h][b].z, v[h][b].w};
      const int off = label - (vb0 + b) * 64 - lane8 * 8;
      uint32_t o[4];
      auto entries = [&](auto far) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float lo = dz_of<CODE, decltype(far)::value>(w[i] & 0xFFFFu, row);
          float hi = dz_of<CODE, decltype(far)::value>(w[i] >> 16, row);
          lo = off == 2 * i ? st.w : lo;
          hi = off == 2 * i + 1 ? st.w : hi;
          o[i] = pack_bf16x2(lo, hi);
        }
      };
      if constexpr (CODE == CE_CODE_SPLIT) {
        const uint32_t most = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
        if (max(most & 0xFFFFu, most >> 16) >= CE_SPLIT_CODE) entries(std::true_type{}); else entries(std::false_type{});
      } else {
        entries(std::true_type{});
      }
      dz[(size_t(vb0 + b) * rows_pad + r) * 8 + lane8] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// ------------------------------------------------------------------ split sums ---
// grad_H of a chunk from its fp32 partials, summed in split order, each row to its position.
__global__ void __launch_bounds__(256)
    kd_ce_split_kernel(const float4* __restrict__ parts, int splits, int64_t stride4, int64_t d4,
                       const int32_t* __restrict__ list, const int32_t* __restrict__ n_valid, int64_t c0, int cap,
                       void* __restrict__ out, int out_bf16) {
  const int64_t n = chunk_rows(n_valid, c0, cap);
  for (int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; i < n * d4; i += int64_t(gridDim.x) * blockDim.x) {
    const int64_t r = i / d4, o = int64_t(list[c0 + r]) * d4 + (i - r * d4);
    float4 a = parts[i];
    for (int sp = 1; sp < splits; ++sp) {
      const float4 b = parts[sp * stride4 + i];
      a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
    }
    if (out_bf16) reinterpret_cast<uint2*>(out)[o] = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
    else reinterpret_cast<float4*>(out)[o] = a;
  }
}

// ------------------------------------------------------------------ scaling ---
// x *= *g, nothing at all where g is 1 (the gradients of a loss that nothing follows).
template <class T>
__global__ void __launch_bounds__(256) kd_ce_scale_kernel(T* __restrict__ x, int64_t n, const float* __restrict__ g) {
  const float f = *g;
  if (f == 1.f) return;
  constexpr int E = 16 / sizeof(T);
  for (int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; i < n / E; i += int64_t(gridDim.x) * blockDim.x) {
    uint4 v = reinterpret_cast<uint4*>(x)[i];
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = sizeof(T) == 4 ? __float_as_uint(__uint_as_float(w[j]) * f)
                            : pack_bf16x2(__uint_as_float(w[j] << 16) * f, __uint_as_float(w[j] & 0xFFFF0000u) * f);
    reinterpret_cast<uint4*>(x)[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ------------------------------------------------------------------ host side ---

// The fp32 partials of grad_H's splits.
size_t ce_split_bytes(int64_t rows_pad, int64_t d) { return align_up(size_t(KD_MAX_SPLITS) * rows_pad * size_t(d) * 4, 256); }

struct CeLayout {
  size_t alpha, list, losses, labels, stats, partials, hidden, dz, kept, gh_part, total;
  int64_t rows_pad, nvb;
  int tiles;
};

// Up to `kept`: what a forward pass that keeps its logits leaves for the gradients; behind it, what they need besides.
CeLayout ce_layout(int64_t N, int64_t d, int64_t V, int64_t chunk, bool step) {
  CeLayout L{};
  const int64_t c = chunk < N ? chunk : N;
  L.rows_pad = (c + BM - 1) / BM * BM;
  L.tiles = int((V + CE_COLS - 1) / CE_COLS);
  L.nvb = (V + 63) / 64;
  size_t off = sizeof(Ctrl);
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  L.alpha = take(4);
  L.list = take(size_t(N) * 4);
  L.losses = take(size_t(N) * 4);
  L.labels = take(size_t(L.rows_pad) * 4);
  L.stats = take(size_t(L.rows_pad) * 16);
  L.partials = take(size_t(L.tiles) * L.rows_pad * 16);
  L.hidden = take(size_t(L.rows_pad) * size_t(d) * 2);
  if (step) {
    L.dz = take(size_t(L.nvb) * L.rows_pad * 128);
    L.kept = off;
    L.gh_part = take(ce_split_bytes(L.rows_pad, d));
  }
  L.total = off;
  return L;
}

struct CeCall {
  const void *H, *W;
  const int32_t* labels;
  const uint8_t* mask;
  int64_t N, d, V, chunk;
  float smooth, z_loss, softcap;
  int ignore;
  const float* grad_loss;
  float *loss, *lse, *losses;
  void* grad_H;
  int grad_H_f32;
  void* grad_W;
  int w_kind;
  void* ws;
  size_t ws_bytes;
  void* split;  // the partials of grad_H's splits
  void *control, *stream;
};

enum CeWhat : int {
  CE_LOSS,   // the loss
  CE_KEEP,   // the loss, the workspace kept as the gradients need it
  CE_STEP,   // the loss and the gradients
};

#define KD_TRY(call)                      \
  do {                                    \
    if ((call) != cudaSuccess) return KD_ERR_CUDA; \
  } while (0)

// Splits of grad_H's reduction over the vocabulary.  In units of one 64-deep k-block of a tile (0.27 us):
// the waves of tiles, each with about 8 blocks of ramp and epilogue, and for a split the reading of its fp32
// partials and one more launch.  8 k-blocks are the least that pays for a split.
int ce_splits(const GemmProblem& q, int slots, int k_blocks) {
  const int64_t tiles = int64_t((q.m_tiles + q.cluster - 1) / q.cluster) * q.n_tiles;
  const double part = double(q.M) * q.N * 4 / 6.5e6 / 0.27;
  int best = 1;
  double best_cost = 1e300;
  for (int S = 1; S <= KD_MAX_SPLITS; ++S) {
    if (S > 1 && k_blocks / S < 8) break;
    const double waves = double((tiles * S + slots - 1) / slots);
    const double cost = waves * (double(k_blocks) / S + 8) + (S > 1 ? S * part + 11 : 0);
    if (cost < best_cost) {
      best_cost = cost;
      best = S;
    }
  }
  return best;
}

// A chunk's gradients: dZ from its kept logits, where they lie, and the two products of dZ and the gathered hidden states.
int ce_gradients(const CeCall& a, const CeLayout& L, uint8_t* w8, int64_t c0, int n, cudaStream_t s) {
  Ctrl* ctrl = static_cast<Ctrl*>(a.ws);
  uint32_t* err = &static_cast<Ctrl*>(a.control)->err;
  const int32_t* list = reinterpret_cast<const int32_t*>(w8 + L.list);
  float* alpha = reinterpret_cast<float*>(w8 + L.alpha);
  const CeCode code = ce_code(a.softcap);
  auto* dz_kernel = code == CE_CODE_DIST   ? kd_ce_dz_kernel<CE_CODE_DIST>
                    : code == CE_CODE_EDGE ? kd_ce_dz_kernel<CE_CODE_EDGE>
                                           : kd_ce_dz_kernel<CE_CODE_SPLIT>;
  prof_before("kd_ce_dz", s);
  dz_kernel<<<unsigned((n + DQ_ROWS - 1) / DQ_ROWS) * unsigned(L.tiles), 256, 0, s>>>(
      reinterpret_cast<uint4*>(w8 + L.dz), int(L.rows_pad), L.nvb, reinterpret_cast<const float4*>(w8 + L.partials),
      int((n + BM - 1) / BM * BM), reinterpret_cast<const float4*>(w8 + L.stats),
      reinterpret_cast<const int32_t*>(w8 + L.labels), &ctrl->n_valid, c0, n, a.softcap, a.grad_loss, 1.f - a.smooth, alpha);
  prof_after(s);
  KD_TRY(cudaGetLastError());

  const uint16_t* Hc = reinterpret_cast<const uint16_t*>(w8 + L.hidden);
  const void* dz = w8 + L.dz;
  const uint64_t d = uint64_t(a.d), V = uint64_t(a.V), row_bytes = d * 2;
  const int grid = gemm_max_grid();
  const bool d64 = a.d % 64 == 0;
  alignas(64) CUtensorMap ta, tb, tc;

  // grad_H = dZ W  (dZ K-major over the vocabulary, W with d contiguous)
  GemmProblem q{};
  q.M = n; q.N = int(a.d); q.K = int(a.V);
  q.b_mn = 1; q.epi = EPI_STORE; q.a_blocked = 1;
  q.m_tiles = (n + BM - 1) / BM;
  q.n_tiles = int((a.d + BN - 1) / BN);
  q.n_group = 1;
  set_cluster(q);
  q.k_splits = ce_splits(q, grid / q.cluster, int((a.V + BK - 1) / BK));
  q.n_units = ((q.m_tiles + q.cluster - 1) / q.cluster) * q.n_tiles * q.k_splits;
  q.rows = n; q.rows_dev = &ctrl->n_valid; q.row_first = int(c0);
  q.err = err;
  q.alpha = alpha;
  q.ldc = a.d;
  if (q.k_splits == 1) {
    q.C = a.grad_H;
    q.c_bf16 = a.grad_H_f32 ? 0 : 1;
    q.row_map = list + c0;
    q.map_rows = a.N;
  } else {
    q.C = a.split;  // fp32 partial per split, summed in split order below
    q.split_stride = L.rows_pad * a.d;
  }
  q.b_box2 = q.cta_pair && d64;
  const int kq = q.cta_pair ? pair_kblocks(0, 1) : 1;
  if (!make_tmap_dz_blocked(&ta, dz, uint64_t(n), uint64_t(L.rows_pad), uint64_t(L.nvb), BM, uint32_t(kq)) ||
      !(q.b_box2 ? make_tmap_mn2_bf16(&tb, a.W, d, V, row_bytes, uint32_t(BK * kq))
                 : make_tmap_2d_bf16(&tb, a.W, d, V, row_bytes, 64, uint32_t(BK * kq))))
    return KD_ERR_CUDA;
  KD_TRY(launch_gemm(q, ta, tb, tb, grid, s));
  if (q.k_splits > 1) {
    const int64_t work = (int64_t(n) * (a.d / 4) + 255) / 256;
    prof_before("kd_ce_split", s);
    kd_ce_split_kernel<<<unsigned(work < 4 * grid ? work : 4 * grid), 256, 0, s>>>(
        static_cast<const float4*>(a.split), q.k_splits, L.rows_pad * a.d / 4, a.d / 4, list,
        &ctrl->n_valid, c0, n, a.grad_H, a.grad_H_f32 ? 0 : 1);
    prof_after(s);
    KD_TRY(cudaGetLastError());
  }

  // grad_W (+)= dZ^T H  (dZ with the vocabulary contiguous, H with d contiguous)
  GemmProblem r{};
  r.M = int(a.V); r.N = int(a.d); r.K = n;
  r.a_mn = r.b_mn = 1; r.a_blocked = 1;
  r.epi = (a.w_kind != KD_GRAD_ADD_F32 && c0 == 0) ? EPI_STORE : EPI_ACCUM;
  r.m_tiles = int((a.V + BM - 1) / BM);
  r.n_tiles = int((a.d + BN - 1) / BN);
  r.n_group = 1;
  r.k_splits = 1;
  set_cluster(r);
  r.n_units = ((r.m_tiles + r.cluster - 1) / r.cluster) * r.n_tiles;
  r.rows = n; r.rows_dev = &ctrl->n_valid; r.row_first = int(c0);
  r.C = a.grad_W; r.ldc = a.d; r.err = err;
  r.alpha = alpha;
  r.c_bf16 = r.c_tma = a.w_kind == KD_GRAD_STORE_BF16;
  r.b_box2 = r.cta_pair && d64;
  const int kr = r.cta_pair ? pair_kblocks(1, 1) : 1;
  if (!(r.cta_pair ? make_tmap_dz_blocked(&ta, dz, uint64_t(n), uint64_t(L.rows_pad), uint64_t(L.nvb),
                                          uint32_t(BK * kr), 2)
                   : make_tmap_dz_blocked(&ta, dz, uint64_t(n), uint64_t(L.rows_pad), uint64_t(L.nvb), BK)) ||
      !(r.b_box2 ? make_tmap_mn2_bf16(&tb, Hc, d, uint64_t(n), row_bytes, uint32_t(BK * kr))
                 : make_tmap_2d_bf16(&tb, Hc, d, uint64_t(n), row_bytes, 64, uint32_t(BK * kr))) ||
      !(r.c_bf16 ? make_tmap_2d_bf16(&tc, a.grad_W, d, V, row_bytes, 64, 32)
                 : make_tmap_2d_f32(&tc, a.grad_W, d, V, d * 4, 32, 32)))
    return KD_ERR_CUDA;
  KD_TRY(launch_gemm(r, ta, tb, tc, grid, s));
  return KD_OK;
}

bool ok4(const void* p) { return p != nullptr && aligned(p, 4); }

kd_status ce_check_options(const CeCall& a) {
  if (!(a.smooth >= 0.f && a.smooth < 1.f) || !(a.z_loss >= 0.f && isfinite(a.z_loss)) ||
      !(a.softcap == 0.f || (a.softcap >= kMinSoftcap && isfinite(a.softcap))))
    return KD_ERR_INVALID_ARG;
  return KD_OK;
}

kd_status ce_check_gradients(const CeCall& a) {
  if (!aligned(a.grad_loss, 4) || !a.grad_H || !aligned(a.grad_H, 16) || !a.grad_W || !aligned(a.grad_W, 16))
    return KD_ERR_INVALID_ARG;
  if (a.w_kind < KD_GRAD_ADD_F32 || a.w_kind > KD_GRAD_STORE_BF16) return KD_ERR_INVALID_ARG;
  if (a.w_kind == KD_GRAD_STORE_BF16 && a.N > a.chunk) return KD_ERR_INVALID_ARG;
  return KD_OK;
}

// A single chunk for all N positions.
int64_t one_chunk(int64_t N) { return N <= KD_MAX_EXTENT ? (N + BM - 1) / BM * BM : BM; }

// Tells what was kept for these sizes and options from anything else; not 0.
uint32_t ce_tag(const CeCall& a) {
  uint32_t smooth, cap, h = 2166136261u;
  memcpy(&smooth, &a.smooth, 4);
  memcpy(&cap, &a.softcap, 4);
  for (uint32_t x : {uint32_t(a.N), uint32_t(a.d), uint32_t(a.V), smooth, cap})
    for (int b = 0; b < 32; b += 8) h = (h ^ (x >> b & 255u)) * 16777619u;
  return h | 1u;
}

int ce_run(CeCall a, CeWhat what) {
  kd_status st = check_proj_args(a.H, a.W, a.N, a.d, a.V, a.chunk, 1.f);
  if (st == KD_OK) st = ce_check_options(a);
  if (st != KD_OK) return st;
  if (!ok4(a.labels) || !ok4(a.loss) || !ok4(a.lse) || !aligned(a.losses, 4)) return KD_ERR_INVALID_ARG;
  if (what == CE_STEP && (st = ce_check_gradients(a)) != KD_OK) return st;
  const CeLayout L = ce_layout(a.N, a.d, a.V, a.chunk, what != CE_LOSS);
  if (!a.ws || !aligned(a.ws, 256) || a.ws_bytes < (what == CE_KEEP ? L.kept : L.total) || !a.control ||
      !aligned(a.control, 256))
    return KD_ERR_WORKSPACE;
  if ((st = check_device()) != KD_OK) return st;

  cudaStream_t s = static_cast<cudaStream_t>(a.stream);
  uint8_t* w8 = static_cast<uint8_t*>(a.ws);
  a.split = w8 + L.gh_part;
  Ctrl* ctrl = static_cast<Ctrl*>(a.ws);
  uint32_t* err = &static_cast<Ctrl*>(a.control)->err;
  int32_t* list = reinterpret_cast<int32_t*>(w8 + L.list);
  float* losses = a.losses ? a.losses : reinterpret_cast<float*>(w8 + L.losses);
  int32_t* labels_c = reinterpret_cast<int32_t*>(w8 + L.labels);
  float4* partials = reinterpret_cast<float4*>(w8 + L.partials);
  uint16_t* Hc = reinterpret_cast<uint16_t*>(w8 + L.hidden);
  const uint64_t d = uint64_t(a.d), V = uint64_t(a.V), row_bytes = d * 2;
  const bool d64 = a.d % 64 == 0;  // two k-blocks per box for CTA pairs
  const int grid = gemm_max_grid();

  prof_before("kd_ce_list", s);
  kd_ce_list_kernel<<<1, LIST_THREADS, 0, s>>>(a.labels, a.mask, a.N, a.ignore, list, &ctrl->n_valid, a.lse, losses,
                                             &ctrl->kept, what == CE_KEEP ? ce_tag(a) : 0u);
  prof_after(s);
  KD_TRY(cudaGetLastError());

  for (int64_t c0 = 0; c0 < a.N; c0 += a.chunk) {
    const int n = int((a.N - c0) < a.chunk ? (a.N - c0) : a.chunk);  // at most
    const bool zero = what == CE_STEP && c0 == 0;
    const int64_t warps = (zero && a.N > L.rows_pad ? a.N : L.rows_pad);
    const int64_t blocks = (warps + GATHER_WARPS - 1) / GATHER_WARPS;
    prof_before("kd_ce_gather", s);
    kd_ce_gather_kernel<<<unsigned(blocks < 8 * grid ? blocks : 8 * grid), GATHER_WARPS * 32, 0, s>>>(
        static_cast<const uint16_t*>(a.H), a.labels, a.mask, a.N, a.d, a.ignore, list, &ctrl->n_valid, c0, n,
        int(L.rows_pad), Hc, labels_c, zero ? a.grad_H : nullptr, a.d * (a.grad_H_f32 ? 4 : 2) / 16, err);
    prof_after(s);
    KD_TRY(cudaGetLastError());

    alignas(64) CUtensorMap th, tw, tq;
    GemmProblem p{};
    p.M = n; p.N = int(a.V); p.K = int(a.d);
    // (the loss alone has no codes: caps that need no series take the kernel with the fewer registers, 509 x 1000 x
    // 50257 with c = 30 91 us a call, 100 with the other)
    p.epi = EPI_CE + (what == CE_LOSS && a.softcap > 0.f && a.softcap <= CE_CAP_NEAR ? CE_CODE_EDGE : ce_code(a.softcap));
    p.m_tiles = (n + BM - 1) / BM;
    p.n_tiles = int((a.V + BN - 1) / BN);
    p.n_group = 1;
    p.k_splits = 1;
    set_cluster(p);
    p.n_units = ((p.m_tiles + p.cluster - 1) / p.cluster) * p.n_tiles;
    p.partials = partials;
    p.rows = n; p.rows_dev = &ctrl->n_valid; p.row_first = int(c0);
    p.tokens = labels_c;
    p.ce_cap = a.softcap;
    p.ce_sum = a.smooth > 0.f;
    p.ce_q = what != CE_LOSS;
    p.err = err;
    p.a_k3d = p.b_k3d = p.cta_pair && d64;
    if (!(p.a_k3d ? make_tmap_mn2_bf16(&th, Hc, d, uint64_t(n), row_bytes, BM)
                  : make_tmap_2d_bf16(&th, Hc, d, uint64_t(n), row_bytes, BK, BM)) ||
        !(p.b_k3d ? make_tmap_mn2_bf16(&tw, a.W, d, V, row_bytes, BN / 2)
                  : make_tmap_2d_bf16(&tw, a.W, d, V, row_bytes, BK, p.cta_pair ? BN / 2 : BN)))
      return KD_ERR_CUDA;
    if (p.ce_q && !make_tmap_dz_blocked(&tq, w8 + L.dz, uint64_t(n), uint64_t(L.rows_pad), uint64_t(L.nvb), 32))
      return KD_ERR_CUDA;
    KD_TRY(launch_gemm(p, th, tw, p.ce_q ? tq : tw, grid, s));

    CeCombine c{};
    c.partials = partials;
    c.tiles = L.tiles; c.rows_pad = int((n + BM - 1) / BM * BM); c.cap = n;
    c.c0 = c0; c.N = a.N; c.V = a.V;
    c.list = list; c.n_valid = &ctrl->n_valid; c.labels_c = labels_c;
    c.smooth = a.smooth; c.z_loss = a.z_loss; c.softcap = a.softcap;
    c.lse = a.lse; c.losses = losses;
    c.row_stats = what != CE_LOSS ? reinterpret_cast<float4*>(w8 + L.stats) : nullptr;
    c.err = err;
    prof_before("kd_ce_combine", s);
    kd_ce_combine_kernel<<<unsigned((n + CC_ROWS - 1) / CC_ROWS), dim3(CC_ROWS, CC_PHASES), 0, s>>>(c);
    prof_after(s);
    KD_TRY(cudaGetLastError());
    if (what == CE_STEP && (st = kd_status(ce_gradients(a, L, w8, c0, n, s))) != KD_OK) return st;
  }
  return map_cuda(launch_loss_reduce(losses, nullptr, a.N, &ctrl->n_valid, a.loss, s));
}

// The gradients of a forward pass (CE_KEEP) from its workspace.
int ce_from_kept(CeCall a) {
  kd_status st = check_proj_args(a.W, a.W, a.N, a.d, a.V, a.chunk, 1.f);  // the hidden states are among what was kept
  if (st == KD_OK) st = ce_check_options(a);
  if (st == KD_OK) st = ce_check_gradients(a);
  if (st != KD_OK) return st;
  const CeLayout L = ce_layout(a.N, a.d, a.V, a.chunk, true);
  if (!a.ws || !aligned(a.ws, 256) || a.ws_bytes < L.kept || !a.split || !aligned(a.split, 256) || !a.control ||
      !aligned(a.control, 256))
    return KD_ERR_WORKSPACE;
  if ((st = check_device()) != KD_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(a.stream);
  const int64_t vecs = a.N * a.d * (a.grad_H_f32 ? 4 : 2) / 16, blocks = (vecs + 255) / 256, most = 8 * gemm_max_grid();
  prof_before("kd_ce_begin", s);
  kd_ce_begin_kernel<<<unsigned(blocks < most ? blocks : most), 256, 0, s>>>(
      static_cast<Ctrl*>(a.ws), ce_tag(a), static_cast<uint4*>(a.grad_H), vecs, &static_cast<Ctrl*>(a.control)->err);
  prof_after(s);
  KD_TRY(cudaGetLastError());
  return ce_gradients(a, L, static_cast<uint8_t*>(a.ws), 0, int(a.N), s);
}

}  // namespace

}  // namespace kd

using namespace kd;

extern "C" {

size_t kd_fused_cross_entropy_workspace(int64_t N, int64_t d, int64_t V, int64_t chunk, int step) {
  if (N < 1 || d < 1 || V < 1 || chunk < 1) return 0;
  return ce_layout(N, d, V, chunk, step != 0).total;
}

int kd_fused_cross_entropy_fwd(const void* H_bf16, const void* W_bf16, const int32_t* labels, const uint8_t* mask,
                               int64_t N, int64_t d, int64_t V, int64_t chunk, float label_smoothing, float z_loss,
                               float softcap, int ignore_index, float* loss_out, float* lse_out,
                               float* loss_per_token_out, void* ws, size_t ws_bytes, void* control, void* stream) {
  CeCall a{};
  a.H = H_bf16; a.W = W_bf16; a.labels = labels; a.mask = mask;
  a.N = N; a.d = d; a.V = V; a.chunk = chunk;
  a.smooth = label_smoothing; a.z_loss = z_loss; a.softcap = softcap; a.ignore = ignore_index;
  a.loss = loss_out; a.lse = lse_out; a.losses = loss_per_token_out;
  a.ws = ws; a.ws_bytes = ws_bytes; a.control = control; a.stream = stream;
  return ce_run(a, CE_LOSS);
}

int kd_fused_cross_entropy_step(const void* H_bf16, const void* W_bf16, const int32_t* labels, const uint8_t* mask,
                                int64_t N, int64_t d, int64_t V, int64_t chunk, float label_smoothing, float z_loss,
                                float softcap, int ignore_index, const float* grad_loss, float* loss_out,
                                float* lse_out, float* loss_per_token_out, void* grad_H, int grad_H_is_fp32,
                                void* grad_W, int grad_W_kind, void* ws, size_t ws_bytes, void* control,
                                void* stream) {
  CeCall a{};
  a.H = H_bf16; a.W = W_bf16; a.labels = labels; a.mask = mask;
  a.N = N; a.d = d; a.V = V; a.chunk = chunk;
  a.smooth = label_smoothing; a.z_loss = z_loss; a.softcap = softcap; a.ignore = ignore_index;
  a.grad_loss = grad_loss;
  a.loss = loss_out; a.lse = lse_out; a.losses = loss_per_token_out;
  a.grad_H = grad_H; a.grad_H_f32 = grad_H_is_fp32; a.grad_W = grad_W; a.w_kind = grad_W_kind;
  a.ws = ws; a.ws_bytes = ws_bytes; a.control = control; a.stream = stream;
  return ce_run(a, CE_STEP);
}

size_t kd_fused_cross_entropy_kept(int64_t N, int64_t d, int64_t V) {
  if (N < 1 || d < 1 || V < 1) return 0;
  return ce_layout(N, d, V, one_chunk(N), true).kept;
}

int kd_fused_cross_entropy_keep(const void* H_bf16, const void* W_bf16, const int32_t* labels, const uint8_t* mask,
                                int64_t N, int64_t d, int64_t V, float label_smoothing, float z_loss, float softcap,
                                int ignore_index, float* loss_out, float* lse_out, float* loss_per_token_out,
                                void* kept, size_t kept_bytes, void* control, void* stream) {
  CeCall a{};
  a.H = H_bf16; a.W = W_bf16; a.labels = labels; a.mask = mask;
  a.N = N; a.d = d; a.V = V; a.chunk = one_chunk(N);
  a.smooth = label_smoothing; a.z_loss = z_loss; a.softcap = softcap; a.ignore = ignore_index;
  a.loss = loss_out; a.lse = lse_out; a.losses = loss_per_token_out;
  a.ws = kept; a.ws_bytes = kept_bytes; a.control = control; a.stream = stream;
  return ce_run(a, CE_KEEP);
}

size_t kd_fused_cross_entropy_bwd_workspace(int64_t N, int64_t d, int64_t V) {
  if (N < 1 || d < 1 || V < 1) return 0;
  return ce_split_bytes(one_chunk(N), d);
}

int kd_fused_cross_entropy_bwd(const void* W_bf16, int64_t N, int64_t d, int64_t V, float label_smoothing,
                               float softcap, const float* grad_loss, void* grad_H, int grad_H_is_fp32, void* grad_W,
                               int grad_W_kind, void* kept, size_t kept_bytes, void* ws, size_t ws_bytes, void* control,
                               void* stream) {
  CeCall a{};
  a.W = W_bf16;
  a.N = N; a.d = d; a.V = V; a.chunk = one_chunk(N);
  a.smooth = label_smoothing; a.softcap = softcap; a.grad_loss = grad_loss;
  a.grad_H = grad_H; a.grad_H_f32 = grad_H_is_fp32; a.grad_W = grad_W; a.w_kind = grad_W_kind;
  a.ws = kept; a.ws_bytes = kept_bytes; a.control = control; a.stream = stream;
  a.split = ws_bytes >= kd_fused_cross_entropy_bwd_workspace(N, d, V) ? ws : nullptr;
  return ce_from_kept(a);
}

int kd_scale_gradient(void* x, int64_t n, int is_fp32, const float* factor, void* stream) {
  if (n < 8 || n % 8 != 0 || !x || !aligned(x, 16) || !ok4(factor)) return KD_ERR_INVALID_ARG;
  kd_status st = check_device();
  if (st != KD_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t blocks = (n / (is_fp32 ? 4 : 8) + 255) / 256, most = 8 * gemm_max_grid();
  prof_before("kd_ce_scale", s);
  if (is_fp32)
    kd_ce_scale_kernel<<<unsigned(blocks < most ? blocks : most), 256, 0, s>>>(static_cast<float*>(x), n, factor);
  else
    kd_ce_scale_kernel<<<unsigned(blocks < most ? blocks : most), 256, 0, s>>>(static_cast<uint16_t*>(x), n, factor);
  prof_after(s);
  return map_cuda(cudaGetLastError());
}

}  // extern "C"
