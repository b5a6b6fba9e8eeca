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
// pass reads and writes each once (2 N V elements).  Both are bound by HBM.  Measured, bf16:
// 4096 x 151936 with the entropy and 5 alternatives 0.211 ms (5.9 TB/s, 87 % of the copy
// bandwidth; fp16 the same; the softmax terms' issue slots and the joins of a row are the rest), its
// gradient 0.376 ms (6.6 TB/s, 98 %); 2048 x 151936 fp32 0.230 ms (5.4 TB/s, 80 %); one row of 201088
// logits 4.4 us, with 20 alternatives 9.2 us.
#include "kd_rows.cuh"

namespace kd {

constexpr int LP_THREADS = 256;      // forward
constexpr int LP_WARPS = LP_THREADS / 32;
constexpr int LP_PER_SM = 6;         // blocks on an SM (4096 x 151936, an earlier loop: 222 us; 4: 232, 5: 229)
constexpr int LP_SLOTS = 32;         // group maxima kept per thread
constexpr int LP_CAND = 1024;        // candidates for the top alternatives
constexpr int LP_LIST = 512;         // groups that may hold one
constexpr int LP_MAX_CLUSTER = 16;
constexpr int LB_THREADS = 256;      // backward
constexpr int LB_PER_SM = 4;

// ------------------------------------------------------------ alternatives ---
// The n largest elements of a row, exactly, without selecting while it streams by.  While the
// row is read each thread keeps the largest element of every group of vectors it reads (it
// needs those maxima for the softmax anyway) and its largest of all, m.  In each of w warps
// the ceil(n / w)-th largest m is reached by that many elements, so the smallest of the w,
// the floor, is reached by at least n: the n largest elements all reach it, and they lie in
// the few groups whose maximum does.  Those groups alone are read again, each vector by a
// thread of its own, so that their latency is paid once.
// Each element's rank key is unique, (value, ~id), so the order is the id's on ties, and a
// candidate's place is the number of candidates above it.  When ties or a crowded row bring
// more candidates than the buffer holds, the row is counted and collected directly.
// In a cluster of c each CTA does this for its share, and sends the first one the keys of its list
// from a bound on: the row's n-th key is at least every share's n-th, and at least the smallest
// of the shares' ceil(n / c)-th.

struct TopState {
  unsigned long long cand[LP_CAND];
  int count;
  int groups;
  int merged;              // in the first CTA: keys that the cluster sent
  unsigned long long sorted[KD_MAX_TOP];
  uint32_t list[LP_LIST];  // slot * LP_THREADS + thread
};

__device__ __forceinline__ unsigned long long rank_key(float x, int64_t col) {
  return (static_cast<unsigned long long>(order_key(x)) << 32) | uint32_t(~uint32_t(col));
}

// Key of the n-th largest (n <= 32) of the lanes' values.
__device__ __forceinline__ uint32_t warp_nth_key(float x, int n) {
  uint32_t key = order_key(x), top = 0;
  for (int i = 0; i < n; ++i) {
    top = __reduce_max_sync(0xffffffffu, key);
    const uint32_t who = __ballot_sync(0xffffffffu, key == top);
    if ((threadIdx.x & 31) == uint32_t(__ffs(who) - 1)) key = 0;  // one of them is taken out
  }
  return top;
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

// The n largest of vectors [lo, hi) when more than LP_CAND elements reach the floor (a key that
// at least n elements reach): the elements above a key T that fewer than n elements exceed, then
// the first ones equal to T by column.
template <int DT>
__device__ void collect_crowded(const Row<DT>& row, int lo, int hi, int n, uint32_t floor, TopState& ts, int* sh) {
  uint32_t T = floor;  // the same in every thread, and so are the counts: all take the same branches
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
    if (order_key(x) > T) {
      const int at = atomicAdd(&ts.count, 1);  // fewer than n of them, but in a row of NaNs
      if (at < LP_CAND) ts.cand[at] = rank_key(x, c);
    }
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
  int V, M, top;
  const int32_t* tokens;
  const uint8_t* mask;
  float tau, k;  // k = log2(e) / tau
  float *logp, *lse, *entropy;
  int32_t* top_ids;
  float* top_logp;
  uint32_t* err;
};

struct LpShared {
  RowStats warp[LP_WARPS];
  uint32_t nth[LP_WARPS];
  // written by the CTAs of the row's cluster (each its own entry)
  RowStats part[LP_MAX_CLUSTER];
  unsigned long long nth_key[LP_MAX_CLUSTER], part_key[LP_MAX_CLUSTER];  // the share's n-th, ceil(n / c)-th
  int scratch[32];
};

// One cluster per row (a single CTA where there are rows enough to fill the GPU): each CTA
// streams its share of the row's vectors; the first one puts the results together.
template <int DT, bool ENT, bool TOP>
__global__ void __launch_bounds__(LP_THREADS, LP_PER_SM) kd_logprobs_fwd_kernel(const LogprobArgs a) {
  extern __shared__ __align__(16) uint8_t lp_smem[];
  __shared__ LpShared sh;
  __shared__ TopState ts;
  constexpr int VE = Elt<DT>::kVec;
  const uint32_t ctas = cluster_size(), rank = cluster_ctarank();
  const int64_t r = blockIdx.x / ctas;
  const int tid = int(threadIdx.x);
  if (a.mask && a.mask[r] == 0) {  // the whole cluster leaves
    if (rank != 0) return;
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
  const int share = (row.nv + int(ctas) - 1) / int(ctas);
  const int lo = min(int(rank) * share, row.nv), hi = min(lo + share, row.nv);
  if (TOP && tid == 0) ts.count = ts.groups = ts.merged = 0;
  __syncwarp();
  if (ctas > 1) cluster_arrive();  // waited for before the first access to another CTA

  // the first CTA's given tokens: their logits are on their way while the row streams by
  int32_t id = 0;
  float z_id = 0.f;
  auto token = [&](int j) {
    id = a.tokens[r * a.M + j];
    if (id >= 0 && id < a.V) z_id = row.at(id);
  };
  if (rank == 0 && tid < a.M) token(tid);

  float* slot_max = reinterpret_cast<float*>(lp_smem);  // [slots][LP_THREADS]
  const int body_lo = max(lo, row.full_lo), body_hi = max(body_lo, min(hi, row.full_hi));
  constexpr int STEP = ROW_GROUP * LP_THREADS;
  const int rounds = (body_hi - body_lo + STEP - 1) / STEP;
  int shift = 0;  // 2^shift rounds share a slot
  while (((rounds - 1) >> shift) >= LP_SLOTS) ++shift;
  RowStats st = stats_empty();
  float running = -INFINITY;
  stream_stats<DT, ENT, LP_THREADS>(
      row, lo, hi, a.k, st, LoadOnce(), [](uint4&, int) {},
      [&](int round, float g) {
        if (!TOP) return;
        running = fmaxf(running, g);  // a NaN leaves it: such a row has no order
        if (KD_DCHECK((round >> shift) < LP_SLOTS, a.err, 0x7601)) slot_max[(round >> shift) * LP_THREADS + tid] = running;
        if (((round + 1) & ((1 << shift) - 1)) == 0) running = -INFINITY;
      });
  const float own_max = st.m;

  // ---- the block's statistics and floor
  stats_block_put<ENT>(st, a.k, sh.warp);
  const int full_warps = min(LP_WARPS, (body_hi - body_lo) / 32);  // every lane has a vector
  const int nth = full_warps ? (a.top + full_warps - 1) / full_warps : 33;
  if (TOP && nth <= 32 && tid / 32 < full_warps) {
    const uint32_t key = warp_nth_key(own_max, nth);
    if ((tid & 31) == 0) sh.nth[tid / 32] = key;
  }
  __syncthreads();
  st = stats_block_get<LP_THREADS, ENT>(a.k, sh.warp);
  uint32_t floor = 0;  // reached by everything
  if (TOP && nth <= 32) {
    floor = 0xFFFFFFFFu;
    for (int w = 0; w < full_warps; ++w) floor = min(floor, sh.nth[w]);
  }

  // ---- the share's candidates, and in a cluster its n largest
  if (TOP) {
    const float floor_v = floor ? order_value(floor) : -INFINITY;
    auto test = [&](int i) {
      float x[VE];
      unpack_vec<DT>(row.load(i), x);
      const int64_t c0 = row.col(i);
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (x[e] >= floor_v && c0 + e >= 0 && c0 + e < row.V) {
          const int at = atomicAdd(&ts.count, 1);
          if (at < LP_CAND) ts.cand[at] = rank_key(x[e], c0 + e);
        }
    };
    if (own_max >= floor_v) {
      // the slots that this thread has written: the last one's rounds may have no vector for it
      const int slots = rounds > 0 ? ((rounds - 1) >> shift) + 1 : 0;
      const int own = body_lo + (slots - 1) * (STEP << shift) + tid < body_hi ? slots : slots - 1;
      for (int q = 0; q < own; ++q)
        if (slot_max[q * LP_THREADS + tid] >= floor_v) {
          const int at = atomicAdd(&ts.groups, 1);
          if (at < LP_LIST) ts.list[at] = uint32_t(q * LP_THREADS + tid);
        }
      const int edge = tid == 0 ? 0 : row.nv - 1;
      if (tid < 2 && edge >= lo && edge < hi && !row.whole(edge) && (tid == 0 || edge != 0)) test(edge);
    }
    __syncthreads();
    const int groups = ts.groups;
    if (groups <= LP_LIST) {
      const int vec_bits = 2 + shift;  // vectors of a group
      static_assert(ROW_GROUP == 4, "a group's vectors as bits");
      for (int w = tid; w < groups << vec_bits; w += LP_THREADS) {
        const uint32_t g = ts.list[w >> vec_bits];
        const int in_group = w & ((1 << vec_bits) - 1);
        const int round = (int(g / LP_THREADS) << shift) + in_group / ROW_GROUP;
        const int i = body_lo + round * STEP + (in_group % ROW_GROUP) * LP_THREADS + int(g % LP_THREADS);
        if (i < body_hi) test(i);
      }
    }
    __syncthreads();
    if (groups > LP_LIST || ts.count > LP_CAND)  // starts with a barrier
      collect_crowded<DT>(row, lo, hi, a.top, floor, ts, sh.scratch);
    if (ctas > 1) {
      for (int j = tid; j < a.top; j += LP_THREADS) ts.sorted[j] = 0;
      __syncthreads();
      const int c = min(ts.count, LP_CAND);
      for (int i = tid; i < c; i += LP_THREADS) {
        const unsigned long long mine = ts.cand[i];
        int place = 0;
        for (int j = 0; j < c; ++j) place += ts.cand[j] > mine;
        if (place < a.top) ts.sorted[place] = mine;
      }
      __syncthreads();
    }
  }

  // ---- the row's
  unsigned long long bound = 0;
  if (ctas > 1) {
    cluster_wait();
    if (tid < int(ctas) && (TOP || tid == 0)) {
      LpShared* other = cluster_map(&sh, uint32_t(tid));
      other->part[rank] = st;
      if (TOP) {
        other->nth_key[rank] = ts.sorted[a.top - 1];
        other->part_key[rank] = ts.sorted[(a.top - 1) / int(ctas)];
      }
    }
    cluster_sync();
    if (!TOP && rank != 0) return;
    st = stats_empty();
    const int lane = tid & (LP_MAX_CLUSTER - 1);
    if (lane < int(ctas)) st = sh.part[lane];
    stats_warp<ENT>(st, a.k, LP_MAX_CLUSTER);
    if (TOP) {
      unsigned long long least = ~0ull;
      for (uint32_t q = 0; q < ctas; ++q) {
        bound = max(bound, sh.nth_key[q]);
        least = min(least, sh.part_key[q]);
      }
      bound = max(bound, least);
    }
  }
  const bool empty = st.s == 0.f;  // every logit is -inf
  const bool odd = st.s != st.s;   // a NaN or +inf logit
  const float log2_s = odd ? st.s : log2f(st.s);
  auto logp_of = [&](float x) { return empty ? -INFINITY : stats_logp(x, st.m, log2_s, a.k, a.tau); };
  if (rank == 0) {
    for (int j = tid; j < a.M; j += LP_THREADS) {
      if (j != tid) token(j);
      float lp;
      if (id < 0 || id >= a.V) {
        raise_error(a.err, KD_DEVERR_BAD_ID, uint32_t(r));
        lp = __int_as_float(0x7FC00000);
      } else {
        lp = logp_of(z_id);
      }
      a.logp[r * a.M + j] = lp;
    }
    if (tid == 0) {
      a.lse[r] = empty ? -INFINITY : stats_lse(st.m, log2_s, a.k, a.tau);
      if (ENT) a.entropy[r] = empty ? 0.f : kLn2 * (log2_s - st.u / st.s);
    }
  }
  if (!TOP) return;

  // ---- the alternatives
  const unsigned long long* keys = ts.cand;
  int c = min(ts.count, LP_CAND);
  if (ctas > 1) {
    unsigned long long* merged = reinterpret_cast<unsigned long long*>(lp_smem);  // the maxima have served
    for (int j = tid; j < a.top; j += LP_THREADS) {
      const unsigned long long key = ts.sorted[j];
      if (key != 0 && key >= bound) {
        const int at = atomicAdd(cluster_map(&ts.merged, 0), 1);
        if (KD_DCHECK(at < int(ctas) * a.top, a.err, 0x7602)) cluster_map(merged, 0)[at] = key;
      }
    }
    cluster_sync();
    if (rank != 0) return;
    keys = merged;
    c = ts.merged;
  }
  if (odd) {
    for (int j = tid; j < a.top; j += LP_THREADS) {
      a.top_ids[r * a.top + j] = j;
      a.top_logp[r * a.top + j] = st.s;
    }
    return;
  }
  for (int i = tid; i < c; i += LP_THREADS) {
    const unsigned long long mine = keys[i];
    int place = 0;
    for (int j = 0; j < c; ++j) place += keys[j] > mine;
    if (place < a.top) {
      a.top_ids[r * a.top + place] = int32_t(~uint32_t(mine));
      a.top_logp[r * a.top + place] = logp_of(order_value(uint32_t(mine >> 32)));
    }
  }
}

// CTAs per row: one where the rows alone give every SM its blocks; otherwise as many as
// would, up to the largest cluster, while each thread still has two groups of vectors (1 x 201088:
// 6.8 us, without clusters 18.7; 128 x 151936 with 5 alternatives 18.5, 26.7; 512 rows 35).
static int logprobs_cluster(int64_t N, int64_t nv) {
  const int64_t want = int64_t(gemm_max_grid()) * LP_PER_SM;
  int c = 1;
  while (c < LP_MAX_CLUSTER && 2 * N * c <= want && nv >= int64_t(2 * c) * ROW_GROUP * LP_THREADS) c *= 2;
  return c;
}

template <int DT, bool ENT, bool TOP>
static cudaError_t logprobs_fwd_one(const LogprobArgs& a, cudaStream_t s) {
  static PerDevice<int> wide;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int v = 0;
  const auto kernel = kd_logprobs_fwd_kernel<DT, ENT, TOP>;
  const int rc = wide.get(dev, &v, [&](int, int* out) {  // clusters of more than 8 CTAs are opted into
    *out = 1;
    return int(cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
  });
  if (rc != 0) return rc > 0 ? cudaError_t(rc) : cudaErrorInvalidDevice;
  const int64_t nv = (int64_t(a.V) + Elt<DT>::kVec - 1) / Elt<DT>::kVec;
  const int ctas = logprobs_cluster(a.N, nv);
  const int64_t rounds = ((nv + 1 + ctas - 1) / ctas + ROW_GROUP * LP_THREADS - 1) / (ROW_GROUP * LP_THREADS);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(ctas);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(unsigned(a.N * ctas), 1, 1);
  cfg.blockDim = dim3(LP_THREADS, 1, 1);
  const size_t maxima = size_t(rounds < LP_SLOTS ? rounds : LP_SLOTS) * LP_THREADS * sizeof(float);
  const size_t merged = ctas > 1 ? size_t(ctas) * a.top * 8 : 0;  // fewer keys than this reach the first CTA
  cfg.dynamicSmemBytes = TOP ? (maxima > merged ? maxima : merged) : 0;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

cudaError_t launch_logprobs_fwd(const void* z, int dtype, int64_t N, int64_t V, int64_t ld, const int32_t* tokens,
                                int M, const uint8_t* mask, float tau, int top, float* logp, float* lse,
                                float* entropy, int32_t* top_ids, float* top_logp, uint32_t* err, cudaStream_t s) {
  LogprobArgs a{};
  a.z = z; a.N = N; a.ld = ld; a.V = int(V); a.M = M; a.top = top;
  a.tokens = tokens; a.mask = mask; a.tau = tau; a.k = log2e_over_tau(tau);
  a.logp = logp; a.lse = lse; a.entropy = entropy; a.top_ids = top_ids; a.top_logp = top_logp; a.err = err;
  cudaError_t e;
  prof_before("kd_logprobs_fwd", s);
  KD_DISPATCH_TYPE(dtype, {
    if (top) e = entropy ? logprobs_fwd_one<DT, true, true>(a, s) : logprobs_fwd_one<DT, false, true>(a, s);
    else e = entropy ? logprobs_fwd_one<DT, true, false>(a, s) : logprobs_fwd_one<DT, false, false>(a, s);
  });
  prof_after(s);
  return e;
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
__global__ void __launch_bounds__(LB_THREADS, LB_PER_SM) kd_logprobs_bwd_kernel(const LogprobGradArgs a) {
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
  auto no_gradient = [&] {  // padding, or every logit -inf
    const float zero[Elt<DT>::kVec] = {};
    for (int i = lo + tid; i < hi; i += LB_THREADS) out.store(i, in.lead, zero);
  };
  if (a.mask && a.mask[r] == 0) {
    no_gradient();
    return;
  }
  float gsum = 0.f;
  for (int j = tid; j < a.M; j += LB_THREADS) {
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
  const float G = sum_block<LB_THREADS>(gsum, sh_sum);  // its barrier: ids, gs, zs written, logits read
  const float h = a.g_ent ? a.g_ent[r] : 0.f;
  // log2 p = (x - base) k - off - log2_s
  float base = 0.f, off = a.lse[r] * kLog2e, log2_s = 0.f;
  if (fabsf(a.lse[r]) > 1024.f) {
    // fp32 holds a logsumexp this large to 1e-4 or worse (or not at all: -inf may be an overflow, of a
    // row of a type's lowest value at tau < 1): take the row's maximum and sum again
    RowStats st = stats_empty();
    stream_stats<DT, false, LB_THREADS>(in, 0, in.nv, a.k, st, LoadOnce(), [](uint4&, int) {}, [](int, float) {});
    __shared__ RowStats sh_stats[LB_THREADS / 32];
    // its barrier: the row is read before any of it is written
    st = stats_block<LB_THREADS, false>(st, a.k, sh_stats);
    if (st.s == 0.f) {
      no_gradient();
      return;
    }
    const bool plain = stats_plain(st.m, a.k);
    base = plain ? 0.f : st.m;
    off = plain ? __fmul_rn(st.m, a.k) : 0.f;
    log2_s = log2f(st.s);
  }
  const float c0 = -(G + (h != 0.f ? h * a.entropy[r] : 0.f)) * a.inv_tau, c1 = -h * kLn2 * a.inv_tau;
  // p (c0 + c1 log2 p); where p is 0 the second factor is kept finite
  auto grad = [&](float x) {
    const float t = fmaf(x - base, a.k, -off) - log2_s;
    return ex2_approx(t) * fmaf(c1, fmaxf(t, -200.f), c0);
  };
  constexpr int VE = Elt<DT>::kVec;
  if (base == 0.f && log2_s == 0.f) {
    const uint64_t k2 = pack2(a.k, a.k), off2 = pack2(-off, -off), c02 = pack2(c0, c0), c12 = pack2(c1, c1);
    stream_map<DT, LB_THREADS>(in, out, lo, hi, [&](float (&x)[VE]) {
#pragma unroll
      for (int e = 0; e < VE; e += 2) {
        float t0, t1;
        unpack2(fma2(pack2(x[e], x[e + 1]), k2, off2), t0, t1);
        const uint64_t p2 = pack2(ex2_approx(t0), ex2_approx(t1));
        unpack2(mul2(p2, fma2(c12, pack2(fmaxf(t0, -200.f), fmaxf(t1, -200.f)), c02)), x[e], x[e + 1]);
      }
    });
  } else {
    stream_map<DT, LB_THREADS>(in, out, lo, hi, [&](float (&x)[VE]) {
#pragma unroll
      for (int e = 0; e < VE; ++e) x[e] = grad(x[e]);
    });
  }
  __syncthreads();
  for (int j = tid; j < a.M; j += LB_THREADS) {
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
  a.tokens = tokens; a.mask = mask; a.inv_tau = inverse_tau(tau); a.k = log2e_over_tau(tau);
  a.lse = lse; a.entropy = entropy; a.g_logp = g_logp; a.g_ent = g_ent; a.err = err;
  // blocks per row: more than one where the rows alone leave SMs idle, while each thread keeps two
  // groups of vectors; one in place, since a block may have to read the whole row first
  const int64_t nv = V / (dtype == KD_F32 ? 4 : 8);
  a.slices = 1;
  while (dz != z && N * a.slices < int64_t(LB_PER_SM) * gemm_max_grid() &&
         nv >= int64_t(4) * a.slices * ROW_GROUP * LB_THREADS)
    a.slices *= 2;
  prof_before("kd_logprobs_bwd", s);
  KD_DISPATCH_TYPE(dtype, kd_logprobs_bwd_kernel<DT><<<unsigned(N * a.slices), LB_THREADS, size_t(M) * 12, s>>>(a));
  prof_after(s);
  return cudaGetLastError();
}

// ---------------------------------------------------- few hidden states ---
// The same scores straight from one or two hidden states (fused_logprobs with a large head): z_v =
// H W_v^T is then bound by reading W once, V d elements.  A warp takes FEW_VOCAB rows of W at a time,
// a lane 16 bytes of each in turn, sums the products over the lanes and keeps running statistics of
// the logits; a block leaves one partial per hidden state, as the projection engine's epilogue does
// per tile.
// Measured, whole calls, V = 201088, d = 2880 (1.16 GB): one row 190 us (6.1 TB/s, 90 % of the copy
// bandwidth), two 209.  One row with three blocks on an SM 3 % slower, with four 15 %.

constexpr int FEW_THREADS = 256;
constexpr int FEW_VOCAB = 4;
constexpr int FEW_PER_SM = 2;  // blocks on an SM

template <int R>
__global__ void __launch_bounds__(FEW_THREADS, FEW_PER_SM)
    kd_logprob_few_kernel(const uint16_t* __restrict__ H, const uint16_t* __restrict__ W, int rows, int d, int64_t V,
                          const int32_t* __restrict__ tokens, const uint8_t* __restrict__ mask, float k,
                          float4* __restrict__ partials, int rows_pad) {
  extern __shared__ __align__(16) float few_h[];  // [R][d] hidden states
  __shared__ RowStats sh[R][FEW_THREADS / 32];
  __shared__ float z_token[R];
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < R * d; i += FEW_THREADS)
    few_h[i] = i < rows * d ? __uint_as_float(uint32_t(H[i]) << 16) : 0.f;
  if (tid < R) z_token[tid] = 0.f;
  int64_t want[R];  // the given tokens (a padding row's is not looked at)
#pragma unroll
  for (int r = 0; r < R; ++r) want[r] = r < rows && (mask == nullptr || mask[r] != 0) ? tokens[r] : -1;
  __syncthreads();
  RowStats st[R];
#pragma unroll
  for (int r = 0; r < R; ++r) st[r] = stats_empty();
  const int nv = d / 8;  // 16-byte vectors of a row (d is a multiple of 8)
  const int64_t warps = int64_t(gridDim.x) * (FEW_THREADS / 32);
  for (int64_t v0 = (int64_t(blockIdx.x) * (FEW_THREADS / 32) + warp) * FEW_VOCAB; v0 < V; v0 += warps * FEW_VOCAB) {
    float acc[FEW_VOCAB][R] = {};
    const uint4* w[FEW_VOCAB];
#pragma unroll
    for (int q = 0; q < FEW_VOCAB; ++q)  // past the vocabulary: its last row again, not added below
      w[q] = reinterpret_cast<const uint4*>(W + (v0 + q < V ? v0 + q : V - 1) * d);
#pragma unroll 2
    for (int i = lane; i < nv; i += 32) {
      uint4 x[FEW_VOCAB];
#pragma unroll
      for (int q = 0; q < FEW_VOCAB; ++q) x[q] = __ldcs(w[q] + i);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 a = reinterpret_cast<const float4*>(few_h + r * d)[2 * i];
        const float4 b = reinterpret_cast<const float4*>(few_h + r * d)[2 * i + 1];
#pragma unroll
        for (int q = 0; q < FEW_VOCAB; ++q) {
          float y[8];
          unpack_vec<KD_BF16>(x[q], y);
          float s = acc[q][r];
          s = fmaf(y[0], a.x, s); s = fmaf(y[1], a.y, s); s = fmaf(y[2], a.z, s); s = fmaf(y[3], a.w, s);
          s = fmaf(y[4], b.x, s); s = fmaf(y[5], b.y, s); s = fmaf(y[6], b.z, s); s = fmaf(y[7], b.w, s);
          acc[q][r] = s;
        }
      }
    }
#pragma unroll
    for (int q = 0; q < FEW_VOCAB; ++q)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float z = warp_sum(acc[q][r]);
        if (lane == 0 && v0 + q < V) {
          if (v0 + q == want[r]) z_token[r] = z;
          if (!(z <= st[r].m)) {
            if (z != z) st[r].s = z;
            else stats_rescale(st[r], z, k);
          }
          const float t = stats_t(z, st[r].m, k), p = ex2_approx(t);
          st[r].s += p;
          st[r].u = fmaf(p, fmaxf(t, -200.f), st[r].u);
        }
      }
  }
  if (lane == 0) {
#pragma unroll
    for (int r = 0; r < R; ++r) sh[r][warp] = st[r];
  }
  __syncthreads();
  if (warp < R && warp < rows) {
    RowStats s = lane < FEW_THREADS / 32 ? sh[warp][lane] : stats_empty();
    stats_warp<true>(s, k);
    if (lane == 0)
      partials[size_t(blockIdx.x) * rows_pad + warp] =
          make_float4(s.m, s.s, z_token[warp], s.u);
  }
}

cudaError_t launch_logprob_few(const uint16_t* H, const uint16_t* W, int rows, int d, int64_t V, const int32_t* tokens,
                               const uint8_t* mask, float tau, float4* partials, int max_units, int* units,
                               cudaStream_t s) {
  const int64_t per_block = FEW_VOCAB * (FEW_THREADS / 32);
  int64_t grid = (V + per_block - 1) / per_block;
  const int most = gemm_max_grid() * FEW_PER_SM;
  if (grid > most) grid = most;
  if (grid > max_units) grid = max_units;
  *units = int(grid);
  const float k = log2e_over_tau(tau);
  prof_before("kd_logprob_few", s);
  cudaError_t e = cudaSuccess;
#define KD_FEW(R_)                                                                                                   \
  do {                                                                                                               \
    static PerDevice<int> done;                                                                                      \
    e = smem_attr_once(done, reinterpret_cast<const void*>(kd_logprob_few_kernel<R_>), FEW_MAX_SMEM);                \
    if (e == cudaSuccess)                                                                                            \
      kd_logprob_few_kernel<R_><<<unsigned(grid), FEW_THREADS, size_t(R_) * d * 4, s>>>(                             \
          H, W, rows, d, V, tokens, mask, k, partials, BM);                                                                \
  } while (0)
  if (rows == 1) KD_FEW(1);
  else KD_FEW(2);
  static_assert(FEW_ROWS == 2, "instances");
#undef KD_FEW
  prof_after(s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kd
