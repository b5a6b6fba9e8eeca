// Log probabilities of given tokens, entropy and top alternatives of dense logits, and the
// gradient of the first two.  With x = z / tau over the V logits of a position:
//   lse   = logsumexp(x)
//   logp_m = x[token_m] - lse
//   H     = lse - sum_v p_v x_v,   p = softmax(x)
//   top   : the n largest logits, equal ones by ascending id, as log probabilities
//   dz_v  = (1 / tau) (sum_m g_m [v = token_m] - p_v (sum_m g_m + h (ln p_v + H)))
// g, h the gradients that reach logp and H.
//
// The forward pass reads each logit once: what it must move is N V elements.  The backward
// pass reads and writes each once (2 N V elements).  Both are bound by HBM.
#include "kd_rows.cuh"

namespace kd {

constexpr int LP_THREADS = 512;
constexpr int LP_SLOTS = 16;      // group maxima kept per thread
constexpr int LP_CAND = 1024;     // candidates for the top alternatives

// ------------------------------------------------------------ alternatives ---
// The n largest elements of a row, exactly, without selecting while it streams by.  While the
// row is read each thread keeps the largest element of every group of vectors it reads (it
// needs those maxima for the softmax anyway) and its largest of all.  At least n elements
// reach the n-th largest of the threads' maxima, T, so the n largest elements all reach T, and
// they lie in the few groups whose maximum reaches T: those groups alone are read again.
// Each element's rank key is unique, (value, ~id), so the order is the id's on ties, and a
// candidate's place is the number of candidates above it.  When ties or a crowded row bring
// more candidates than the buffer holds, the row is counted and collected directly.

struct TopState {
  unsigned long long cand[LP_CAND];
  int count;
  uint32_t floor;   // key that at least n elements reach
};

__device__ __forceinline__ unsigned long long rank_key(float x, int64_t col) {
  return (static_cast<unsigned long long>(order_key(x)) << 32) | uint32_t(~uint32_t(col));
}

// Warp 0: a key that at least n of the THREADS values reach (n <= THREADS), and few more.
template <int THREADS>
__device__ __forceinline__ uint32_t warp_floor(const float* vals, int n) {
  constexpr int E = THREADS / 32;
  const int lane = threadIdx.x & 31;
  uint32_t key[E], lo = 0xFFFFFFFFu, hi = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    key[i] = order_key(vals[i * 32 + lane]);
    lo = min(lo, key[i]);
    hi = max(hi, key[i]);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lo == hi) return lo;
  ++hi;  // no value reaches hi; all reach lo
  const int enough = n + (n >> 2) + 4;
  while (hi - lo > 1) {
    const uint32_t mid = lo + ((hi - lo) >> 1);
    int c = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) c += key[i] >= mid;
    c = __reduce_add_sync(0xffffffffu, c);
    if (c >= n) {
      lo = mid;
      if (c <= enough) break;
    } else {
      hi = mid;
    }
  }
  return lo;
}

// All threads: visit(column, value) for every element of vectors [lo, hi) of the row.
template <int DT, class F>
__device__ __forceinline__ void for_each(const Row<DT>& row, int lo, int hi, F&& visit) {
  for (int i = lo + int(threadIdx.x); i < hi; i += blockDim.x) {
    float x[Elt<DT>::kVec];
    unpack_vec<DT>(row.load(i), x);
    const int64_t c0 = row.col(i);
#pragma unroll
    for (int e = 0; e < Elt<DT>::kVec; ++e)
      if (c0 + e >= 0 && c0 + e < row.V) visit(c0 + e, x[e]);
  }
}

template <int DT>
__device__ int count_reaching(const Row<DT>& row, int lo, int hi, uint32_t key, int* sh) {
  __syncthreads();
  if (threadIdx.x == 0) *sh = 0;
  __syncthreads();
  int c = 0;
  for_each<DT>(row, lo, hi, [&](int64_t, float x) { c += order_key(x) >= key; });
  c = __reduce_add_sync(0xffffffffu, c);
  if ((threadIdx.x & 31) == 0) atomicAdd(sh, c);
  __syncthreads();
  return *sh;
}

// The n largest of vectors [lo, hi) when more than LP_CAND elements reach the floor: elements
// above a key T that fewer than n elements exceed, then the first ones equal to T by column.
template <int DT>
__device__ void collect_crowded(const Row<DT>& row, int lo, int hi, int n, TopState& ts, int* sh) {
  uint32_t T = ts.floor;
  if (count_reaching<DT>(row, lo, hi, T + 1, sh) >= n) {
    uint32_t a = T, b = 0xFFFFFFFFu;  // count(a) >= n; nothing reaches b
    while (b - a > 1) {
      const uint32_t mid = a + ((b - a) >> 1);
      if (count_reaching<DT>(row, lo, hi, mid, sh) >= n) a = mid;
      else b = mid;
    }
    T = a;
  }
  __syncthreads();
  if (threadIdx.x == 0) ts.count = 0;
  __syncthreads();
  for_each<DT>(row, lo, hi, [&](int64_t c, float x) {
    if (order_key(x) > T) ts.cand[atomicAdd(&ts.count, 1)] = rank_key(x, c);  // fewer than n of them
  });
  __syncthreads();
  // columns in ascending order, a block's width at a time, until n are found
  const int64_t c_lo = row.col(lo) < 0 ? 0 : row.col(lo);
  const int64_t c_hi = row.col(hi) < row.V ? row.col(hi) : row.V;
  for (int64_t c0 = c_lo; c0 < c_hi; c0 += blockDim.x) {
    const int have = ts.count;  // the same in every thread: nothing is added before the barrier
    if (have >= n) break;
    const int64_t c = c0 + threadIdx.x;
    float x = 0.f;
    bool eq = false;
    if (c < c_hi) {
      x = row.at(c);
      eq = order_key(x) == T;
    }
    const uint32_t ballot = __ballot_sync(0xffffffffu, eq);
    int* per_warp = sh;  // [32]
    if ((threadIdx.x & 31) == 0) per_warp[threadIdx.x >> 5] = __popc(ballot);
    __syncthreads();
    int before = have, all = 0;
    for (int w = 0; w < int(blockDim.x >> 5); ++w) {
      if (w < int(threadIdx.x >> 5)) before += per_warp[w];
      all += per_warp[w];
    }
    const int at = before + __popc(ballot & ((1u << (threadIdx.x & 31)) - 1u));
    if (eq && at < n) ts.cand[at] = rank_key(x, c);
    __syncthreads();
    if (threadIdx.x == 0) ts.count = min(n, have + all);
    __syncthreads();
  }
}

// ------------------------------------------------------------------ forward ---

struct LogprobArgs {
  const void* z;
  int64_t N, ld;
  int V, M, top, dtype;
  const int32_t* tokens;
  const uint8_t* mask;
  float tau, k;  // k = log2(e) / tau
  float *logp, *lse, *entropy;
  int32_t* top_ids;
  float* top_logp;
  uint32_t* err;
};

// One block per row.
template <int DT, bool ENT, bool TOP>
__global__ void __launch_bounds__(LP_THREADS) kd_logprobs_fwd_kernel(const LogprobArgs a) {
  extern __shared__ __align__(16) uint8_t lp_smem[];
  __shared__ RowStats sh_stats[32];
  __shared__ float sh_max[LP_THREADS];
  __shared__ int sh_int[32];
  const int64_t r = blockIdx.x;
  const int tid = int(threadIdx.x);
  if (a.mask && a.mask[r] == 0) {
    for (int j = tid; j < a.M; j += LP_THREADS) a.logp[r * a.M + j] = 0.f;
    if (TOP)
      for (int j = tid; j < a.top; j += LP_THREADS) {
        a.top_ids[r * a.top + j] = 0;
        a.top_logp[r * a.top + j] = 0.f;
      }
    if (tid == 0) {
      a.lse[r] = 0.f;
      if (ENT) a.entropy[r] = 0.f;
    }
    return;
  }
  const Row<DT> row(static_cast<const typename Elt<DT>::raw*>(a.z) + r * a.ld, a.V);

  float* gmax_sh = reinterpret_cast<float*>(lp_smem);  // [slots][LP_THREADS]
  const int per_round = ROW_GROUP * LP_THREADS;
  const int rounds = (row.nv + per_round - 1) / per_round;
  const int merge = (rounds + LP_SLOTS - 1) / LP_SLOTS;  // rounds that share a slot
  RowStats st;
  float slot_max = -INFINITY;
  for (int it = 0; it < rounds; ++it) {
    uint4 v[ROW_GROUP];
    row.load_group(v, it * per_round + tid, LP_THREADS, row.nv);
    const float g = group_max<DT>(v);
    if (TOP) {
      slot_max = fmaxf(slot_max, g);
      if ((it + 1) % merge == 0 || it + 1 == rounds) {
        gmax_sh[(it / merge) * LP_THREADS + tid] = slot_max;
        slot_max = -INFINITY;
      }
    }
    stats_add<DT, ENT>(st, v, g, a.k);
  }
  if (TOP) sh_max[tid] = st.m;
  st = stats_block<LP_THREADS>(st, a.k, sh_stats);
  const float ln_s = st.s > 0.f ? logf(st.s) : st.s;  // s = 0: every logit is -inf; NaN stays
  const bool empty = st.s == 0.f;

  for (int j = tid; j < a.M; j += LP_THREADS) {
    const int32_t id = a.tokens[r * a.M + j];
    float lp;
    if (id < 0 || id >= a.V) {
      raise_error(a.err, KD_DEVERR_BAD_ID, uint32_t(r));
      lp = __int_as_float(0x7FC00000);
    } else {
      lp = empty ? -INFINITY : (row.at(id) - st.m) / a.tau - ln_s;
    }
    a.logp[r * a.M + j] = lp;
  }
  if (tid == 0) {
    a.lse[r] = empty ? -INFINITY : st.m / a.tau + ln_s;
    if (ENT) a.entropy[r] = empty ? 0.f : ln_s - kLn2 * (st.u / st.s);
  }
  if (!TOP) return;

  if (st.s != st.s) {  // a NaN or +inf logit: no order to report
    for (int j = tid; j < a.top; j += LP_THREADS) {
      a.top_ids[r * a.top + j] = j;
      a.top_logp[r * a.top + j] = st.s;
    }
    return;
  }
  __shared__ TopState ts;
  if (tid < 32) {
    const uint32_t f = warp_floor<LP_THREADS>(sh_max, a.top);
    if (tid == 0) {
      ts.floor = f;
      ts.count = 0;
    }
  }
  __syncthreads();
  const float floor_v = order_value(ts.floor);
  const int slots = (rounds + merge - 1) / merge;
  for (int q = 0; q < slots; ++q) {
    if (!(gmax_sh[q * LP_THREADS + tid] >= floor_v)) continue;
    const int it_hi = min(rounds, (q + 1) * merge);
    for (int it = q * merge; it < it_hi; ++it) {
      for (int j = 0; j < ROW_GROUP; ++j) {
        const int i = it * per_round + j * LP_THREADS + tid;
        if (i >= row.nv) break;
        float x[Elt<DT>::kVec];
        unpack_vec<DT>(row.load(i), x);
        const int64_t c0 = row.col(i);
#pragma unroll
        for (int e = 0; e < Elt<DT>::kVec; ++e)
          if (x[e] >= floor_v && c0 + e >= 0 && c0 + e < row.V) {
            const int at = atomicAdd(&ts.count, 1);
            if (at < LP_CAND) ts.cand[at] = rank_key(x[e], c0 + e);
          }
      }
    }
  }
  __syncthreads();
  if (ts.count > LP_CAND) collect_crowded<DT>(row, 0, row.nv, a.top, ts, sh_int);
  const int c = ts.count;
  for (int i = tid; i < c; i += LP_THREADS) {
    const unsigned long long mine = ts.cand[i];
    int place = 0;
    for (int j = 0; j < c; ++j) place += ts.cand[j] > mine;
    if (place < a.top) {
      const float x = order_value(uint32_t(mine >> 32));
      a.top_ids[r * a.top + place] = int32_t(~uint32_t(mine));
      a.top_logp[r * a.top + place] = empty ? -INFINITY : (x - st.m) / a.tau - ln_s;
    }
  }
}

size_t logprobs_smem(int V, int dtype) {
  const int64_t vec = dtype == KD_F32 ? 4 : 8;
  const int64_t nv = (int64_t(V) + vec - 1) / vec + 1;
  int64_t rounds = (nv + ROW_GROUP * LP_THREADS - 1) / (ROW_GROUP * LP_THREADS);
  return size_t(rounds < LP_SLOTS ? rounds : LP_SLOTS) * LP_THREADS * sizeof(float);
}

cudaError_t launch_logprobs_fwd(const void* z, int dtype, int64_t N, int64_t V, int64_t ld, const int32_t* tokens,
                                int M, const uint8_t* mask, float tau, int top, float* logp, float* lse,
                                float* entropy, int32_t* top_ids, float* top_logp, uint32_t* err, cudaStream_t s) {
  LogprobArgs a{};
  a.z = z; a.N = N; a.ld = ld; a.V = int(V); a.M = M; a.top = top; a.dtype = dtype;
  a.tokens = tokens; a.mask = mask; a.tau = tau; a.k = float(1.4426950408889634 / double(tau));
  a.logp = logp; a.lse = lse; a.entropy = entropy; a.top_ids = top_ids; a.top_logp = top_logp; a.err = err;
  const size_t smem = top ? logprobs_smem(a.V, dtype) : 0;
  prof_before("kd_logprobs_fwd", s);
  KD_DISPATCH_TYPE(dtype, {
    if (top) {
      if (entropy) kd_logprobs_fwd_kernel<DT, true, true><<<unsigned(N), LP_THREADS, smem, s>>>(a);
      else kd_logprobs_fwd_kernel<DT, false, true><<<unsigned(N), LP_THREADS, smem, s>>>(a);
    } else {
      if (entropy) kd_logprobs_fwd_kernel<DT, true, false><<<unsigned(N), LP_THREADS, 0, s>>>(a);
      else kd_logprobs_fwd_kernel<DT, false, false><<<unsigned(N), LP_THREADS, 0, s>>>(a);
    }
  });
  prof_after(s);
  return cudaGetLastError();
}

// ----------------------------------------------------------------- backward ---

struct LogprobGradArgs {
  const void* z;
  void* dz;
  int64_t N, ld, ld_dz;
  int V, M, slices;
  const int32_t* tokens;
  const uint8_t* mask;
  float inv_tau, k;
  const float *lse, *entropy, *g_logp, *g_ent;
  uint32_t* err;
};

// Block (row, slice of the row's vectors).  dz may be z itself: a block reads the logits of its
// tokens first and rewrites their gradients last, and every vector is read and written by one
// thread.
template <int DT>
__global__ void __launch_bounds__(LP_THREADS) kd_logprobs_bwd_kernel(const LogprobGradArgs a) {
  extern __shared__ __align__(16) uint8_t lp_smem[];
  __shared__ float sh_sum[32];
  int32_t* ids = reinterpret_cast<int32_t*>(lp_smem);     // [M]
  float* gs = reinterpret_cast<float*>(ids + a.M);        // [M]
  float* zs = gs + a.M;                                   // [M]
  const int64_t r = blockIdx.x / unsigned(a.slices);
  const int slice = int(blockIdx.x % unsigned(a.slices));
  const int tid = int(threadIdx.x);
  using raw = typename Elt<DT>::raw;
  const Row<DT> in(static_cast<const raw*>(a.z) + r * a.ld, a.V);
  const Row<DT> out(static_cast<raw*>(a.dz) + r * a.ld_dz, a.V);
  const int per = (in.nv + a.slices - 1) / a.slices;
  const int lo = min(slice * per, in.nv), hi = min(lo + per, in.nv);
  const bool live = (a.mask == nullptr || a.mask[r] != 0) && a.lse[r] != -INFINITY;
  if (!live) {  // padding, or every logit -inf: no gradient
    const float zero[Elt<DT>::kVec] = {};
    for (int i = lo + tid; i < hi; i += LP_THREADS) out.store(i, in.lead, zero);
    return;
  }
  float gsum = 0.f;
  for (int j = tid; j < a.M; j += LP_THREADS) {
    int32_t id = a.tokens[r * a.M + j];
    const float g = a.g_logp[r * a.M + j];
    if (id < 0 || id >= a.V) {
      raise_error(a.err, KD_DEVERR_BAD_ID, uint32_t(r));
      id = -1;
    } else {
      gsum += g;
      const int i = (in.lead + id) / Elt<DT>::kVec;
      if (i >= lo && i < hi) zs[j] = in.at(id);
    }
    ids[j] = id;
    gs[j] = g;
  }
  const float G = sum_block<LP_THREADS>(gsum, sh_sum);  // its barrier: ids, gs, zs written, logits read
  const float h = a.g_ent ? a.g_ent[r] : 0.f;
  // log2 p = (x - base) k - off
  float base = 0.f, off = a.lse[r] * kLog2e;
  if (fabsf(a.lse[r]) > 1024.f) {
    // fp32 holds a logsumexp this large to 1e-4 or worse (a row of a type's lowest value: not at
    // all): take the row's maximum and sum again
    RowStats st;
    for (int i0 = 0; i0 < in.nv; i0 += ROW_GROUP * LP_THREADS) {
      uint4 v[ROW_GROUP];
      in.load_group(v, i0 + tid, LP_THREADS, in.nv);
      stats_add<DT, false>(st, v, group_max<DT>(v), a.k);
    }
    __shared__ RowStats sh_stats[32];
    st = stats_block<LP_THREADS>(st, a.k, sh_stats);  // its barrier: the row is read before any of it is written
    base = st.m;
    off = log2f(st.s);
  }
  const float c0 = -(G + (h != 0.f ? h * a.entropy[r] : 0.f)) * a.inv_tau, c1 = -h * kLn2 * a.inv_tau;
  // p (c0 + c1 log2 p); where p is 0 the second factor is kept finite
  auto grad = [&](float x) {
    const float t = fmaf(x - base, a.k, -off);
    return ex2_approx(t) * fmaf(c1, fmaxf(t, -200.f), c0);
  };
  for (int i0 = lo; i0 < hi; i0 += ROW_GROUP * LP_THREADS) {
    uint4 v[ROW_GROUP];
    in.load_group(v, i0 + tid, LP_THREADS, hi);
#pragma unroll
    for (int j = 0; j < ROW_GROUP; ++j) {
      const int64_t i = int64_t(i0) + tid + j * LP_THREADS;
      if (i >= hi) break;
      float x[Elt<DT>::kVec];
      unpack_vec<DT>(v[j], x);
#pragma unroll
      for (int e = 0; e < Elt<DT>::kVec; ++e) x[e] = grad(x[e]);
      out.store(int(i), in.lead, x);
    }
  }
  __syncthreads();
  for (int j = tid; j < a.M; j += LP_THREADS) {
    const int id = ids[j];
    if (id < 0) continue;
    const int i = (in.lead + id) / Elt<DT>::kVec;
    if (i < lo || i >= hi) continue;
    bool first = true;
    float g = 0.f;
    for (int q = 0; q < a.M; ++q)
      if (ids[q] == id) {
        first &= q >= j;
        g += gs[q];
      }
    if (first) *out.elt(id) = Elt<DT>::narrow(grad(zs[j]) + g * a.inv_tau);
  }
}

cudaError_t launch_logprobs_bwd(const void* z, int dtype, int64_t N, int64_t V, int64_t ld, const int32_t* tokens,
                                int M, const uint8_t* mask, float tau, const float* lse, const float* entropy,
                                const float* g_logp, const float* g_ent, void* dz, int64_t ld_dz, uint32_t* err,
                                cudaStream_t s) {
  LogprobGradArgs a{};
  a.z = z; a.dz = dz; a.N = N; a.ld = ld; a.ld_dz = ld_dz; a.V = int(V); a.M = M;
  a.tokens = tokens; a.mask = mask; a.inv_tau = 1.0f / tau; a.k = float(1.4426950408889634 / double(tau));
  a.lse = lse; a.entropy = entropy; a.g_logp = g_logp; a.g_ent = g_ent; a.err = err;
  a.slices = 1;  // more only where dz is not z: a block may read the whole row
  prof_before("kd_logprobs_bwd", s);
  KD_DISPATCH_TYPE(dtype, kd_logprobs_bwd_kernel<DT><<<unsigned(N), LP_THREADS, size_t(M) * 12, s>>>(a));
  prof_after(s);
  return cudaGetLastError();
}

}  // namespace kd
