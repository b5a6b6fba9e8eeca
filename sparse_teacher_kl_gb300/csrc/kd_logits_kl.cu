// KL(teacher || student) on dense student logits against a teacher's cached top logits, and its
// gradient.  Per position, with x = z / tau, q = softmax(x) over the V logits and S the K cached
// ids:
//   without the rest: p = softmax(t / tau) over S (the mass outside dropped)
//   with the rest   : p_k = exp(t_k / tau - t_lse), p_R = 1 - sum_k p_k >= 0, t_lse the
//                     teacher's logsumexp over its whole vocabulary; every id outside S is one
//                     more class R, q_R = sum of q outside S
//   KL   = sum_k p_k (ln p_k - ln q_k) [+ p_R (ln p_R - ln q_R)]
//   dz_v = c (q_v - p_v) on S;  off S: c q_v, or with the rest c (q_R - p_R) e^(x_v - lse_R),
//          lse_R the logsumexp of x outside S;  c = grad_loss / (N_valid tau)
// q_R is summed over the ids outside S alone (never as 1 - sum of q on S), so it keeps its
// digits however small it is; a bitmap of S over the row's columns keeps S out of that sum.
//
// Loss and gradient in one call must read each logit once and write each gradient once
// (2 N V elements): bound by HBM.
#include "kd_rows.cuh"

namespace kd {

constexpr int LK_THREADS = 512;
constexpr int LK_MAX_SMEM = 200 * 1024;

enum LkMode : int { LK_FWD = 1, LK_BWD = 2, LK_STEP = 3 };

struct LogitsKlArgs {
  const void* z;
  void* dz;
  int64_t N, ld, ld_dz;
  int V, K;
  const int32_t* ids;
  const float* tlog;
  const float* t_lse;     // with the rest class
  const uint8_t* mask;
  float tau, k;           // k = log2(e) / tau
  float4* stats;          // [N] (m, s) of the row and (m, s) outside S
  float* kl;              // [N]
  const float* grad_loss;
  const int32_t* n_valid; // NULL: N
  uint32_t* err;
};

// Shared memory of a row: entries [K] of (id, or -1 where it is absent or
// repeats an earlier one; p; z), and the bitmap of S: one byte per
// vector, one bit per element of it.
static size_t lk_smem(int64_t V, int K, int dtype) {
  const int64_t vec = dtype == KD_F32 ? 4 : 8;
  const int64_t nv = (V + vec - 1) / vec + 1;
  return size_t(K) * 12 + size_t((nv + 15) / 16 * 16);
}

// One block per row.
template <int DT, bool REST, int MODE>
__global__ void __launch_bounds__(LK_THREADS) kd_logits_kl_kernel(const LogitsKlArgs a) {
  extern __shared__ __align__(16) uint8_t lk_raw[];
  __shared__ RowStats sh_stats[32], sh_stats2[32];
  __shared__ float sh_a[32], sh_b[32];
  __shared__ int repeated;
  using raw = typename Elt<DT>::raw;
  constexpr int VE = Elt<DT>::kVec;
  const int64_t r = blockIdx.x;
  const int tid = int(threadIdx.x);
  const Row<DT> in(static_cast<const raw*>(a.z) + r * a.ld, a.V);
  const Row<DT> out(MODE == LK_FWD ? nullptr : static_cast<raw*>(a.dz) + r * a.ld_dz, a.V);
  const float zero[VE] = {};
  if (a.mask && a.mask[r] == 0) {
    if (MODE != LK_BWD && tid == 0) {
      a.kl[r] = 0.f;
      if (MODE == LK_FWD) a.stats[r] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
    }
    if (MODE != LK_FWD)
      for (int i = tid; i < in.nv; i += LK_THREADS) out.store(i, in.lead, zero);
    return;
  }

  // ---- the teacher's entries
  uint32_t* bits = reinterpret_cast<uint32_t*>(lk_raw);  // byte i: vector i
  const int bit_words = (in.nv + 15) / 16 * 4;
  int32_t* ids = reinterpret_cast<int32_t*>(bits + bit_words);
  float* ps = reinterpret_cast<float*>(ids + a.K);
  float* zs = ps + a.K;
  for (int i = tid; i < bit_words; i += LK_THREADS) bits[i] = 0;
  if (tid == 0) repeated = 0;
  const float* tr = a.tlog + r * a.K;
  const int32_t* idr = a.ids + r * a.K;
  float shift = 0.f, log_norm = 0.f;  // ln p_k = (t_k - shift) / tau - log_norm
  if (REST) {
    log_norm = a.t_lse[r];
    __syncthreads();
  } else {
    float tm = -INFINITY;
    for (int j = tid; j < a.K; j += LK_THREADS) tm = fmaxf(tm, tr[j]);
    RowStats t;
    t.m = tm;
    if (tm != -INFINITY)
      for (int j = tid; j < a.K; j += LK_THREADS) t.s += ex2_approx((tr[j] - tm) * a.k);
    t = stats_block<LK_THREADS>(t, a.k, sh_stats2);
    shift = t.m == -INFINITY ? 0.f : t.m;
    log_norm = t.s > 0.f ? logf(t.s) : t.s;
  }
  // an entry of logit -inf is absent: its id is not looked at
  float p_sum = 0.f;
  RowStats ss;  // the student's logits on S, each id once
  for (int j = tid; j < a.K; j += LK_THREADS) {
    const float t = tr[j];
    int32_t id = -1;
    float p = 0.f, z = -INFINITY;
    if (t != -INFINITY) {
      id = idr[j];
      if (id < 0 || id >= a.V) {
        raise_error(a.err, KD_DEVERR_BAD_ID, uint32_t(r));
        id = -1;
      } else {
        p = expf((t - shift) / a.tau - log_norm);
        z = in.at(id);
        const int at = in.lead + id;  // element of the vector grid
        const uint32_t bit = 1u << (((at / VE) & 3) * 8 + at % VE);
        if (atomicOr(&bits[at / (4 * VE)], bit) & bit) {
          repeated = 1;
          id = -1;
        } else if (MODE != LK_BWD && z != -INFINITY) {
          RowStats one;
          one.m = z;
          one.s = 1.f;
          stats_merge(ss, one, a.k);
        }
      }
    }
    ids[j] = id;
    ps[j] = p;
    zs[j] = z;
    p_sum += p;
  }
  p_sum = sum_block<LK_THREADS>(p_sum, sh_a);  // its barrier: entries and bitmap written, z read
  bool rest = REST;  // some id lies outside S
  if (REST && a.K == a.V) {
    float distinct = 0.f;
    for (int j = tid; j < a.K; j += LK_THREADS) distinct += ids[j] >= 0 ? 1.f : 0.f;
    rest = sum_block<LK_THREADS>(distinct, sh_b) < float(a.V);
  }
  const bool teacher = REST || p_sum > 0.f || p_sum != p_sum;

  // ---- the student's statistics
  RowStats st, sr;
  if (MODE != LK_BWD) {
    const uint8_t* bytes = reinterpret_cast<const uint8_t*>(bits);
    for (int i0 = 0; i0 < in.nv; i0 += ROW_GROUP * LK_THREADS) {
      uint4 v[ROW_GROUP];
      in.load_group(v, i0 + tid, LK_THREADS, in.nv);
      if (REST) {
#pragma unroll
        for (int j = 0; j < ROW_GROUP; ++j) {
          const int i = i0 + tid + j * LK_THREADS;
          const uint32_t b = i < in.nv ? bytes[i] : 0u;
          if (b) {  // take the elements of S out
            uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
            for (int e = 0; e < VE; ++e)
              if ((b >> e) & 1u) {
                if (DT == KD_F32) w[e] = Elt<DT>::kNegInf;
                else if (e & 1) w[e >> 1] = (w[e >> 1] & 0xFFFFu) | (Elt<DT>::kNegInf & 0xFFFF0000u);
                else w[e >> 1] = (w[e >> 1] & 0xFFFF0000u) | (Elt<DT>::kNegInf & 0xFFFFu);
              }
            v[j] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      stats_add<DT, false>(st, v, group_max<DT>(v), a.k);
    }
    st = stats_block<LK_THREADS>(st, a.k, sh_stats);
    if (REST) {
      sr = st;
      __syncthreads();  // sh_stats2 may still be read
      ss = stats_block<LK_THREADS>(ss, a.k, sh_stats2);
      stats_merge(st, ss, a.k);
    }
    if (MODE == LK_FWD && tid == 0) a.stats[r] = make_float4(st.m, st.s, sr.m, sr.s);
  } else {
    const float4 q = a.stats[r];
    st.m = q.x; st.s = q.y; sr.m = q.z; sr.s = q.w;
  }
  const bool empty = st.s == 0.f;  // every logit -inf
  const float ln_s = empty ? 0.f : logf(st.s);
  float p_rest = 0.f, log_q_rest = -INFINITY;
  if (REST) {
    if (rest) p_rest = fmaxf(1.f - p_sum, 0.f);
    if (sr.s > 0.f) log_q_rest = (sr.m - st.m) / a.tau + logf(sr.s) - ln_s;
    if (sr.s != sr.s) log_q_rest = sr.s;
  }

  if (MODE != LK_BWD) {
    float kl = 0.f;
    for (int j = tid; j < a.K; j += LK_THREADS)
      if (!(ps[j] <= 0.f)) {
        const float log_q = empty ? -INFINITY : (zs[j] - st.m) / a.tau - ln_s;
        kl = fmaf(ps[j], (tr[j] - shift) / a.tau - log_norm - log_q, kl);
      }
    kl = sum_block<LK_THREADS>(kl, sh_b);
    if (REST && p_rest > 0.f) kl = fmaf(p_rest, logf(p_rest) - log_q_rest, kl);
    if (tid == 0) a.kl[r] = teacher ? kl : 0.f;
  }
  if (MODE == LK_FWD) return;

  // ---- the gradient
  if (empty || !teacher) {
    for (int i = tid; i < in.nv; i += LK_THREADS) out.store(i, in.lead, zero);
    return;
  }
  const int64_t n_valid = a.n_valid ? int64_t(*a.n_valid) : a.N;
  const float c = *a.grad_loss / (float(n_valid) * a.tau);
  const float base = REST ? sr.m : st.m;
  float scale;  // off S: dz = scale 2^((x - base) k)
  if (REST) scale = sr.s > 0.f ? c * (expf(log_q_rest) - p_rest) / sr.s : (sr.s == 0.f ? 0.f : sr.s);
  else scale = c / st.s;
  const float safe = base == -INFINITY ? 0.f : base;  // nothing outside S: every x there is -inf
  for (int i0 = 0; i0 < in.nv; i0 += ROW_GROUP * LK_THREADS) {
    uint4 v[ROW_GROUP];
    in.load_group(v, i0 + tid, LK_THREADS, in.nv);
#pragma unroll
    for (int j = 0; j < ROW_GROUP; ++j) {
      const int64_t i = int64_t(i0) + tid + j * LK_THREADS;
      if (i >= in.nv) break;
      float x[VE];
      unpack_vec<DT>(v[j], x);
#pragma unroll
      for (int e = 0; e < VE; ++e) x[e] = scale * ex2_approx((x[e] - safe) * a.k);
      out.store(int(i), in.lead, x);
    }
  }
  __syncthreads();
  for (int j = tid; j < a.K; j += LK_THREADS) {
    const int id = ids[j];
    if (id < 0) continue;
    float p = ps[j];
    if (repeated) {  // all entries of this id, in their order
      p = 0.f;
      for (int q = 0; q < a.K; ++q)
        if (idr[q] == id && tr[q] != -INFINITY) p += ps[q];
    }
    const float q = expf((zs[j] - st.m) / a.tau - ln_s);
    *out.elt(id) = Elt<DT>::narrow(c * (q - p));
  }
}

template <int MODE>
static cudaError_t lk_launch(const LogitsKlArgs& a, int dtype, size_t smem, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  KD_DISPATCH_TYPE(dtype, {
    static PerDevice<int> done[2];
    if (a.t_lse) {
      e = smem_attr_once(done[1], reinterpret_cast<const void*>(kd_logits_kl_kernel<DT, true, MODE>), LK_MAX_SMEM);
      if (e == cudaSuccess) kd_logits_kl_kernel<DT, true, MODE><<<unsigned(a.N), LK_THREADS, smem, s>>>(a);
    } else {
      e = smem_attr_once(done[0], reinterpret_cast<const void*>(kd_logits_kl_kernel<DT, false, MODE>), LK_MAX_SMEM);
      if (e == cudaSuccess) kd_logits_kl_kernel<DT, false, MODE><<<unsigned(a.N), LK_THREADS, smem, s>>>(a);
    }
  });
  return e != cudaSuccess ? e : cudaGetLastError();
}

bool logits_kl_fits(int64_t V, int K, int dtype) { return lk_smem(V, K, dtype) <= size_t(LK_MAX_SMEM); }

cudaError_t launch_logits_kl(int mode, const void* z, int dtype, int64_t N, int64_t V, int64_t ld, const int32_t* ids,
                             const float* tlog, int K, const float* t_lse, const uint8_t* mask, float tau,
                             float* stats, float* kl, const float* grad_loss, const int32_t* n_valid, void* dz,
                             int64_t ld_dz, uint32_t* err, cudaStream_t s) {
  LogitsKlArgs a{};
  a.z = z; a.dz = dz; a.N = N; a.ld = ld; a.ld_dz = ld_dz; a.V = int(V); a.K = K; a.ids = ids; a.tlog = tlog;
  a.t_lse = t_lse; a.mask = mask; a.tau = tau; a.k = float(1.4426950408889634 / double(tau));
  a.stats = reinterpret_cast<float4*>(stats); a.kl = kl; a.grad_loss = grad_loss; a.n_valid = n_valid; a.err = err;
  const size_t smem = lk_smem(V, K, dtype);
  cudaError_t e;
  prof_before(mode == LK_FWD ? "kd_logits_kl_fwd" : mode == LK_BWD ? "kd_logits_kl_bwd" : "kd_logits_kl_step", s);
  if (mode == LK_FWD) e = lk_launch<LK_FWD>(a, dtype, smem, s);
  else if (mode == LK_BWD) e = lk_launch<LK_BWD>(a, dtype, smem, s);
  else e = lk_launch<LK_STEP>(a, dtype, smem, s);
  prof_after(s);
  return e;
}

}  // namespace kd
