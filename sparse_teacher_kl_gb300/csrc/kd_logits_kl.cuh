// KL(teacher || student) on dense student logits against a teacher's cached top logits, and its
// gradient.  Per position, with x = z / tau, q = softmax(x) over the V logits and S the K cached
// ids:
//   without the rest: p = softmax(t / tau) over S (the mass outside dropped)
//   with the rest   : p_k = exp(t_k / tau - t_lse), p_R = 1 - sum_k p_k (0 where that is below
//                     2^-21 (1 + |t_lse|)), t_lse the teacher's logsumexp over its whole
//                     vocabulary; every id outside S is one more class R, q_R = sum of q outside S
//   KL   = sum_k p_k (ln p_k - ln q_k) [+ p_R (ln p_R - ln q_R)]
//   dz_v = c (q_v - p_v) on S;  off S: c q_v, or with the rest c (q_R - p_R) e^(x_v - lse_R),
//          lse_R the logsumexp of x outside S;  c = grad_loss / (N_valid tau)
// q_R is summed over the ids outside S alone (never as 1 - sum of q on S), so it keeps its
// digits however small it is; a bitmap of S over the row's columns keeps S out of that sum.
//
// Loss and gradient in one call must read each logit once and write each gradient once
// (2 N V elements): bound by HBM.  Measured, bf16, K = 100: 4096 x 201088 with the rest class
// 0.641 ms (5.1 TB/s, 76 % of the copy bandwidth; DRAM reads 12 % over the row's own bytes), 8192 x
// 32000 with 5 % padding 0.211 ms (4.8 TB/s, 71 %); what is left are the joins of a row's
// statistics, where a block's loads run dry.  Tried at 4096 x 201088 and slower: the row kept in
// the shared memory of a cluster by bulk copies (0.83 ms at best, the joins cost more), the next
// row's statistics and this row's gradient in one loop (1.04 ms: too few loads in flight).  Rows
// that fit into one SM were not tried that way; they are read twice like the others.
#pragma once

#include "kd_rows.cuh"

namespace kd {

constexpr int LK_MAX_CLUSTER = 16;
constexpr int LK_MAX_SMEM = 200 * 1024;
constexpr int LKB_THREADS = 256;       // backward
constexpr int LKB_PER_SM = 4;

struct LogitsKlArgs {
  const void* z;
  void* dz;
  int64_t N, ld, ld_dz;
  int V, K;
  int share;    // forward and step: at least the vectors of a CTA's part of a row
  int slices;   // backward: blocks per row
  const int32_t* ids;
  const float* tlog;
  const float* t_lse;     // with the rest class
  const uint8_t* mask;
  float tau, inv_tau, k;  // k = log2(e) / tau
  float4* stats;          // [N] (m, s) of the row and (m, s) outside S
  float* kl;              // [N]
  const float* grad_loss;
  const int32_t* n_valid; // NULL: N, or in a step with a mask the block counts them
  uint32_t* err;
};

// ------------------------------------------------------------ the teacher ---
// A row's K cached entries are the work of a few warps, a lane each, so that what they cost is
// paid in few instructions beside the row's own.  The block owns elements [e_lo, e_hi) of the
// row's vector grid, and the entries in them.  An entry of logit -inf is absent: its id is not
// looked at.
struct LkEntries {
  uint32_t* bits;   // S within the block's vectors: byte i is vector i, a bit per element
  int32_t* loc;     // [K] element (grid index - e_lo), or -1: absent or another block's;
                    // -2 - element: its id repeats that of another entry
  float* t;         // [K] (t - shift) / tau, shift the row's largest t (0 with the rest class)
  float* e;         // [K] probability, but for the factor 1 / sum
  float* z;         // [K] the student's logit, for entries of this block
};

// Bytes of shared memory for n vectors and K entries.
__host__ __device__ __forceinline__ int64_t lk_entry_bytes(int64_t n, int K) {
  return (n + 15) / 16 * 16 + (int64_t(K) * 16 + 15) / 16 * 16;
}

__device__ __forceinline__ LkEntries lk_entries(uint8_t* at, int n, int K) {
  LkEntries t;
  t.bits = reinterpret_cast<uint32_t*>(at);
  t.loc = reinterpret_cast<int32_t*>(at + (n + 15) / 16 * 16);
  t.t = reinterpret_cast<float*>(t.loc + K);
  t.e = t.t + K;
  t.z = t.e + K;
  return t;
}

// The sums below are of e times this (KD_MAX_K entries of at most 1, so that no sum passes a single
// entry's size: student logits of a type's lowest value on cached ids make entries of up to 3e38).
constexpr float kEntryScale = 1.f / KD_MAX_K;

// What a warp's entries come to.
struct LkSummary {
  float e_sum;             // over all of them
  float s_m, s_s;          // the student's logits on the block's part of S, each id once
  float z_ref, e, d;       // over the block's: sum of e, and of e (t - (z - z_ref) / tau), scaled;
                           // z_ref the largest z (-inf where there is none)
  int distinct, repeats;   // ids that came first, and again
  float t_lse;
};
__device__ __forceinline__ LkSummary lk_nothing() { return {0.f, -INFINITY, 0.f, -INFINITY, 0.f, 0.f, 0, 0, 0.f}; }

struct LkEntryScratch {
  float t_max[4];
  LkSummary warp[4];
  __device__ __forceinline__ bool repeated(int warps) const {
    int n = 0;
    for (int w = 0; w < warps; ++w) n += warp[w].repeats;
    return n != 0;
  }
};

// A thread's first entry, loaded ahead of its use.
struct LkAhead {
  float t, t_lse;
  int32_t id;
};
template <bool REST>
__device__ __forceinline__ LkAhead lk_ahead(const LogitsKlArgs& a, int64_t r, int et) {
  LkAhead p = {-INFINITY, 0.f, -1};
  if (et < a.K) {
    p.t = a.tlog[r * a.K + et];
    p.id = a.ids[r * a.K + et];
  }
  if (REST) p.t_lse = a.t_lse[r];
  return p;
}

// The entries of row r by ET threads (et = 0 .. ET - 1, whole warps, at most four); sync() is a
// barrier among them.  `logit(id, element)` reads the student's logit of an entry of this block.
// Ends with a barrier: summaries in sh.warp.
template <int DT, bool REST, int ET, class Sync, class Logit>
__device__ __forceinline__ void lk_teacher(const LogitsKlArgs& a, int64_t r, const Row<DT>& row, int e_lo, int e_hi,
                                           const LkEntries& t, LkEntryScratch& sh, const LkAhead& ahead, int et,
                                           bool report, Sync&& sync, Logit&& logit) {
  constexpr int VE = Elt<DT>::kVec, EW = ET / 32;
  static_assert(EW <= 4, "scratch");
  const int lane = et & 31, ew = et >> 5;
  auto t_of = [&](int j) { return j == et ? ahead.t : a.tlog[r * a.K + j]; };
  float tm = -INFINITY;
  if (!REST)
    for (int j = et; j < a.K; j += ET) tm = fmaxf(tm, t_of(j));
  const int words = ((e_hi - e_lo) / VE + 15) / 16;
  for (int i = et; i < words; i += ET) reinterpret_cast<uint4*>(t.bits)[i] = make_uint4(0, 0, 0, 0);
  if (!REST) {
    tm = warp_max(tm);
    if (lane == 0) sh.t_max[ew] = tm;
  }
  sync();
  float shift = 0.f;  // with the rest class the normaliser is given
  if (!REST) {
    tm = sh.t_max[0];
#pragma unroll
    for (int w = 1; w < EW; ++w) tm = fmaxf(tm, sh.t_max[w]);
    if (tm != -INFINITY) shift = tm;
  }
  LkSummary o = lk_nothing();
  o.t_lse = ahead.t_lse;
  for (int j = et; j < a.K; j += ET) {
    const float tj = t_of(j);
    int32_t loc = -1;
    float e = 0.f, z = -INFINITY, ts = -INFINITY;
    if (tj != -INFINITY) {
      const int32_t id = j == et ? ahead.id : a.ids[r * a.K + j];
      if (uint32_t(id) >= uint32_t(a.V)) {
        if (report) raise_error(a.err, KD_DEVERR_BAD_ID, uint32_t(r));
      } else {
        ts = (tj - shift) * a.inv_tau;  // the difference first: t / tau may round by more than 1
        e = expf(REST ? ts - ahead.t_lse : ts);
        const int at = row.lead + id - e_lo;
        if (at >= 0 && at < e_hi - e_lo && KD_DCHECK(at / VE / 16 < words, a.err, 0x7701)) {
          const uint32_t bit = 1u << (((at / VE) & 3) * 8 + at % VE);
          if (atomicOr(&t.bits[at / (4 * VE)], bit) & bit) {
            ++o.repeats;
            loc = -2 - at;
          } else {
            loc = at;
            z = logit(id, at);
            ++o.distinct;
          }
        }
      }
    }
    t.loc[j] = loc;
    t.t[j] = ts;
    t.e[j] = e;
    t.z[j] = z;
    o.e_sum += e;
    o.z_ref = fmaxf(o.z_ref, z);
  }
  // the sums relative to the warp's largest logit; only with an entry that repeats an id do they
  // wait for every entry's logit.  An id counts once in S: with its entry that came first to the
  // bitmap or, where there are more, with its lowest one, so that the order of the sum is fixed.
  auto sums = [&](bool repeats) {
    o.z_ref = warp_max(o.z_ref);
    o.s_s = o.e = o.d = 0.f;
    for (int j = et; j < a.K; j += ET) {
      const int loc = t.loc[j];
      if (loc == -1) continue;
      const float z = t.z[j], e = t.e[j];
      bool once = loc >= 0;
      if (repeats) {
        const int at = loc >= 0 ? loc : -2 - loc;
        once = true;
        for (int q = 0; q < j; ++q) once &= t.loc[q] != at && t.loc[q] != -2 - at;
      }
      if (once) {
        if (!(fabsf(z) <= 3.402823466e38f) && z != -INFINITY) o.s_s = __int_as_float(0x7FC00000);  // NaN or +inf
        else if (z != -INFINITY) o.s_s += ex2_approx(stats_t(z, o.z_ref, a.k));
      }
      if (!(e <= 0.f)) {
        const float es = e * kEntryScale;
        o.e += es;
        o.d += z == -INFINITY ? INFINITY : fmaf(-es * a.inv_tau, z - o.z_ref, es * t.t[j]);
      }
    }
    o.s_s = warp_sum(o.s_s);
    o.e = warp_sum(o.e);
    o.d = warp_sum(o.d);
    o.s_m = o.z_ref;
    if (lane == 0) sh.warp[ew] = o;
  };
  o.e_sum = warp_sum(o.e_sum);
  o.distinct = __reduce_add_sync(0xffffffffu, o.distinct);
  o.repeats = __reduce_add_sync(0xffffffffu, o.repeats);
  sums(false);
  sync();
  if (sh.repeated(EW)) {
    sync();  // every thread has read the summaries
    for (int j = et; j < a.K; j += ET)
      if (t.loc[j] < -1) {  // the logit of the entry that came first
        for (int q = 0; q < a.K; ++q)
          if (t.loc[q] == -2 - t.loc[j]) t.z[j] = t.z[q];
        o.z_ref = fmaxf(o.z_ref, t.z[j]);
      }
    __syncwarp();
    sums(true);
    sync();
  }
}

// One warp, whose first lanes hold parts of a row's entries: all of them together.
__device__ __forceinline__ void lk_merge(const LogitsKlArgs& a, LkSummary& o) {
  const float ref = warp_max(o.z_ref);
  o.d = warp_sum(o.z_ref == -INFINITY || o.e == 0.f ? o.d : fmaf(-o.e * a.inv_tau, o.z_ref - ref, o.d));
  o.z_ref = ref;
  o.e = warp_sum(o.e);
  o.e_sum = warp_sum(o.e_sum);
  o.distinct = __reduce_add_sync(0xffffffffu, o.distinct);
  RowStats st = {o.s_m, o.s_s, 0.f};
  stats_warp<false>(st, a.k);
  o.s_m = st.m;
  o.s_s = st.s;
}

// What every thread needs of a row once its statistics are known.
struct LkRow {
  float m, log2_s;            // ln q(x) = stats_logp(x, m, log2_s)
  float inv_sum, log_norm;    // p_k = e_k inv_sum,  ln p_k = t_k - log_norm
  float c, scale, sub, off;   // dz = scale 2^((x - sub) k + off) outside S, c (q - p) on it
  float rest_kl;              // the rest class's term of the divergence
  int empty, none;            // every logit is -inf; nothing cached (without the rest)
};

// From the row's statistics (all of it; outside S): c = grad_loss / (N_valid tau).
template <bool REST>
__device__ __forceinline__ LkRow lk_row(const LogitsKlArgs& a, const RowStats& all, const RowStats& rest,
                                        const LkSummary& t, float t_lse, float c) {
  LkRow w;
  w.m = all.m;
  w.empty = all.s == 0.f;
  w.log2_s = w.empty ? 0.f : log2f(all.s);
  w.c = c;
  w.rest_kl = 0.f;
  w.none = !REST && t.e_sum == 0.f;
  const RowStats& b = REST ? rest : all;
  if (REST) {
    w.log_norm = t_lse;
    w.inv_sum = 1.f;
    // Below the resolution of its inputs a remainder is rounding, not mass (a teacher whose cache holds
    // everything leaves some 1e-6 of either sign, and a student without mass there would be infinitely
    // wrong): t_lse is rounded by |t_lse| 2^-24, t / tau by as much and half more, the exponentials and
    // their sum by 2^-21 in all.  (A teacher row of nothing but -inf has all its mass there, wherever that
    // is: KL 0 and no gradient, as without the rest class.)  The entries may also cover the whole vocabulary (K = V, one block).
    const float left = 1.f - t.e_sum;
    const float least = t_lse == -INFINITY ? 0.f : 4.76837158e-7f * (1.f + fabsf(t_lse));
    const float p_rest = t.distinct == a.V || left < least ? 0.f : left;
    float log_q = -INFINITY;  // of the rest
    if (b.s > 0.f) {
      log_q = kLn2 * (stats_shift(b.m, all.m, a.k) + log2f(b.s) - w.log2_s);
    }
    if (p_rest > 0.f) {
      w.rest_kl = p_rest * (logf(p_rest) - log_q);
      // a logarithm beyond fp32's range, which its share of the mass may bring back into it
      if (log_q == -INFINITY && b.s > 0.f) w.rest_kl = -(p_rest * a.inv_tau) * (b.m - all.m);
    }
    w.scale = b.s == 0.f ? 0.f : c * (expf(log_q) - p_rest) / b.s;
    if (b.s != b.s) w.rest_kl = w.scale = b.s;
  } else {
    w.log_norm = t.e_sum > 0.f ? logf(t.e_sum) : t.e_sum;
    w.inv_sum = 1.f / t.e_sum;
    w.scale = c / b.s;
  }
  const bool plain = stats_plain(b.m, a.k);
  w.sub = plain || b.m == -INFINITY ? 0.f : b.m;  // nothing outside S: every x there is -inf
  w.off = plain ? -__fmul_rn(b.m, a.k) : 0.f;
  return w;
}

// A block's part of the divergence: sum of p (ln p - ln q) over its entries.
__device__ __forceinline__ float lk_kl(const LogitsKlArgs& a, const LkRow& w, float z_ref, float e_here, float d_here) {
  if (w.none || e_here == 0.f) return 0.f;
  if (d_here != d_here) return d_here;
  if (w.empty || z_ref == -INFINITY) return INFINITY;
  const float log_q = stats_logp(z_ref, w.m, w.log2_s, a.k, a.tau);
  return w.inv_sum * (1.f / kEntryScale) * (d_here - e_here * (w.log_norm + log_q));
}

// Vectors [lo, hi) of a row by the block's first THREADS threads: the gradient outside S.
template <int DT, int THREADS>
__device__ __forceinline__ void lk_stream_grad(const Row<DT>& in, const Row<DT>& out, int lo, int hi, float scale,
                                               float sub, float off, float k) {
  constexpr int VE = Elt<DT>::kVec;
  const uint64_t k2 = pack2(k, k), off2 = pack2(off, off), scale2 = pack2(scale, scale);
  auto grad = [&](float (&x)[VE]) {
#pragma unroll
    for (int e = 0; e < VE; e += 2) {
      float t0, t1;
      unpack2(fma2(pack2(x[e], x[e + 1]), k2, off2), t0, t1);
      unpack2(mul2(pack2(ex2_approx(t0), ex2_approx(t1)), scale2), x[e], x[e + 1]);
    }
  };
  if (sub == 0.f)
    stream_map<DT, THREADS>(in, out, lo, hi, grad);
  else  // far from zero: see stats_t
    stream_map<DT, THREADS>(in, out, lo, hi, [&](float (&x)[VE]) {
#pragma unroll
      for (int e = 0; e < VE; ++e) x[e] -= sub;
      grad(x);
    });
}

// dz on S, over the formula's values: one rounding of c (q - p), an id's entries together.
template <int DT>
__device__ __forceinline__ void lk_write_entries(const LogitsKlArgs& a, const Row<DT>& in, const Row<DT>& out, int e_lo,
                                                 const LkEntries& t, const LkRow& w, bool repeated, int first, int step) {
  for (int j = first; j < a.K; j += step) {
    const int loc = t.loc[j];
    if (loc < 0) continue;
    float e = t.e[j];
    if (repeated) {  // all entries of this id, in their order
      e = 0.f;
      for (int q = 0; q < a.K; ++q)
        if (t.loc[q] == loc || t.loc[q] == -2 - loc) e += t.e[q];
    }
    const float log_q = stats_logp(t.z[j], w.m, w.log2_s, a.k, a.tau);
    *out.elt(e_lo + loc - in.lead) = Elt<DT>::narrow(w.c * (expf(log_q) - e * w.inv_sum));
  }
}

template <int DT>
__device__ __forceinline__ void lk_zero(const Row<DT>& in, const Row<DT>& out, int lo, int hi, int first, int step) {
  const float zero[Elt<DT>::kVec] = {};
  for (int i = lo + first; i < hi; i += step) out.store(i, in.lead, zero);
}

// -------------------------------------------------------- forward and step ---
// Persistent blocks, a row at a time (a long row, or one of few: a cluster, each CTA an equal
// share of its vectors).  A step reads a row twice, for the statistics and for the gradient, but
// the second time from L2: the first pass asks L2 to keep the lines, the second gives them up,
// and the rows in flight are kept to half of L2, so that a row crosses HBM once.
//   consumer warps  a row's statistics, then its gradient
//   entry warps     meanwhile the next row's entries (softmax, places, the student's logits
//                   there), and the gradient on S of the row before
// With the rest class the statistics leave S out by its bitmap.  Every wait is bounded.

struct LkPart {
  float4 stats;  // (m, s) outside S (or of all), (m, s) on S
  float4 kl;     // z_ref, e, d
};

struct LkShared {
  uint64_t ready[2], done[2], parts[2];  // of a row's entries; of its gradient; of the cluster's statistics
  RowStats warp[2][32];
  LkPart part[2][LK_MAX_CLUSTER];
  LkEntryScratch entry[2];
  LkRow row[2];
  int valid[32];  // rows counted by each warp
  uint32_t abort_flag;
};

template <int THREADS>
__device__ __forceinline__ void named_sync(int id) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(THREADS) : "memory");
}

template <int DT, bool REST, bool STEP, int CW, int EW, int PER_SM>
__global__ void __launch_bounds__((CW + EW) * 32, PER_SM) kd_logits_kl_kernel(const LogitsKlArgs a) {
  extern __shared__ __align__(16) uint8_t lk_raw[];
  __shared__ LkShared sh;
  using raw = typename Elt<DT>::raw;
  constexpr int VE = Elt<DT>::kVec, CT = CW * 32, ET = EW * 32;
  constexpr uint32_t NI = Elt<DT>::kNegInf;
  static_assert(CW <= 32 && EW <= 4, "LkShared, LkEntryScratch");
  const uint32_t ctas = cluster_size(), rank = cluster_ctarank();
  const int tid = int(threadIdx.x), lane = tid & 31;
  const int64_t first = blockIdx.x / ctas, step = gridDim.x / ctas;
  const int64_t count = first < a.N ? (a.N - first + step - 1) / step : 0;
  const int64_t entry_size = lk_entry_bytes(a.share, a.K);
  const raw* const z = static_cast<const raw*>(a.z);

  if (tid == 0) {
    sh.abort_flag = 0;
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.ready[b], 1);
      mbar_init(&sh.done[b], CW);
      mbar_init(&sh.parts[b], ctas);
    }
    fence_mbar_init();
  }
  __syncthreads();
  if (ctas > 1) cluster_sync();  // every CTA's barriers exist
  // A wait that runs out raises the flag; from then on every wait returns at once: all roles run
  // through their rows (whose results are void) and leave together.
  volatile uint32_t* const stop = &sh.abort_flag;
  // idle_ns: looks at a barrier that is long in coming this often, to leave the issue slots to others.
  auto wait = [&](uint64_t* bar, uint32_t phase, uint32_t where, uint32_t idle_ns = 0) {
    const uint64_t t0 = idle_ns ? globaltimer_ns() : 0;
    while (idle_ns && *stop == 0 && !mbar_try_wait(bar, phase) && globaltimer_ns() - t0 < kWaitLimitNs / 2)
      __nanosleep(idle_ns);
    if (*stop == 0) mbar_wait(bar, phase, stop, a.err, where);
  };
  auto is_live = [&](int64_t r) { return a.mask == nullptr || a.mask[r] != 0; };
  auto share_of = [&](const Row<DT>& row, int& lo, int& hi) {
    const int share = (row.nv + int(ctas) - 1) / int(ctas);
    lo = min(int(rank) * share, row.nv);
    hi = min(lo + share, row.nv);
  };

  if (tid >= CT) {
    // ------------------------------------------------------------ entry warps
    const int et = tid - CT;
    auto sync = [&] { named_sync<ET>(1); };
    LkAhead ahead = {};
    if (count > 0) ahead = lk_ahead<REST>(a, first, et);
    for (int64_t it = 0; it <= count; ++it) {
      if (it < count) {  // row it's entries, while the consumers are at the row before
        const int64_t r = first + it * step;
        const int b = int(it & 1);
        const LkAhead now = ahead;
        if (it + 1 < count) ahead = lk_ahead<REST>(a, r + step, et);
        if (is_live(r)) {
          const Row<DT> row(z + r * a.ld, a.V);
          int lo, hi;
          share_of(row, lo, hi);
          lk_teacher<DT, REST, ET>(a, r, row, lo * VE, hi * VE, lk_entries(lk_raw + b * entry_size, a.share, a.K),
                                   sh.entry[b], now, et, rank == 0, sync,
                                   [&](int id, int) { return row.at(id); });
        } else {
          sync();
        }
        if (et == 0) mbar_arrive(&sh.ready[b]);
      }
      if (it > 0) {  // the gradient on S of the row before
        const int64_t r = first + (it - 1) * step;
        const int b = int((it - 1) & 1);
        wait(&sh.done[b], uint32_t((it - 1) >> 1) & 1u, 0x601u, 500);
        if (STEP && is_live(r) && !sh.row[b].empty && !sh.row[b].none) {
          const Row<DT> in(z + r * a.ld, a.V);
          const Row<DT> out(static_cast<raw*>(a.dz) + r * a.ld_dz, a.V);
          int lo, hi;
          share_of(in, lo, hi);
          lk_write_entries<DT>(a, in, out, lo * VE, lk_entries(lk_raw + b * entry_size, a.share, a.K), sh.row[b],
                               sh.entry[b].repeated(EW), et, ET);
        }
        sync();  // row it + 1's entries take this one's place
      }
    }
  } else {
    // --------------------------------------------------------- consumer warps
    const int warp = tid >> 5;
    float c = 0.f;
    if (STEP) {
      float n_valid = float(a.N);
      if (a.n_valid) {
        n_valid = float(*a.n_valid);
      } else if (a.mask) {
        int n = 0;
        for (int64_t i = tid; i < a.N; i += CT) n += a.mask[i] != 0;
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) sh.valid[warp] = n;
        named_sync<CT>(2);
        n = 0;
        for (int q = 0; q < CW; ++q) n += sh.valid[q];
        n_valid = float(n);
      }
      c = *a.grad_loss * a.inv_tau / n_valid;
    }
    uint32_t exchanges = 0;
    for (int64_t it = 0; it < count; ++it) {
      const int64_t r = first + it * step;
      const int b = int(it & 1);
      const Row<DT> in(z + r * a.ld, a.V);
      const Row<DT> out(STEP ? static_cast<raw*>(a.dz) + r * a.ld_dz : nullptr, a.V);
      int lo, hi;
      share_of(in, lo, hi);
      if (!is_live(r)) {
        if (STEP) lk_zero<DT>(in, out, lo, hi, tid, CT);
        if (rank == 0 && tid == 0) {
          a.kl[r] = 0.f;
          if (!STEP) a.stats[r] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
        }
        wait(&sh.ready[b], uint32_t(it >> 1) & 1u, 0x602u);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.done[b]);
        __syncwarp();
        continue;
      }

      // ---- statistics
      if (REST) wait(&sh.ready[b], uint32_t(it >> 1) & 1u, 0x602u);
      const uint8_t* in_s = lk_raw + b * entry_size;  // the bitmap of S, a byte a vector
      auto without_s = [&](uint4& v, int i) {
        if (!REST || i >= hi) return;
        const uint32_t bits = in_s[i - lo];
        if (bits == 0) return;
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if ((bits >> e) & 1u) {
            if (DT == KD_F32) w[e & 3] = NI;
            else if (e & 1) w[e >> 1] = (w[e >> 1] & 0xFFFFu) | (NI & 0xFFFF0000u);
            else w[e >> 1] = (w[e >> 1] & 0xFFFF0000u) | (NI & 0xFFFFu);
          }
        v = make_uint4(w[0], w[1], w[2], w[3]);
      };
      RowStats st = stats_empty();
      if (STEP) stream_stats<DT, false, CT>(in, lo, hi, a.k, st, LoadKeep(), without_s, [](int, float) {});
      else stream_stats<DT, false, CT>(in, lo, hi, a.k, st, LoadOnce(), without_s, [](int, float) {});
      __syncwarp();
      stats_warp<false>(st, a.k);
      // The wait stands before the write: the row's entries are posted after every consumer warp is done
      // with row it - 2, and so warp 0 has read that row's statistics.  (A padding row between the two has
      // no barrier of the consumers that would say so.)
      if (!REST) wait(&sh.ready[b], uint32_t(it >> 1) & 1u, 0x602u);
      if (lane == 0) sh.warp[b][warp] = st;
      named_sync<CT>(2);
      if (warp == 0) {
        st = lane < CW ? sh.warp[b][lane] : stats_empty();
        stats_warp<false>(st, a.k);
        LkSummary t = lk_nothing();
        if (lane < EW) t = sh.entry[b].warp[lane];
        const float t_lse = sh.entry[b].warp[0].t_lse;
        lk_merge(a, t);
        RowStats on_s = {t.s_m, t.s_s, 0.f};
        float z_ref = t.z_ref, e_here = lane == 0 ? t.e : 0.f, d_here = t.d;
        if (ctas > 1) {
          const uint32_t x = exchanges & 1u;
          if (lane < int(ctas)) {
            LkShared* other = cluster_map(&sh, uint32_t(lane));
            other->part[x][rank].stats = make_float4(st.m, st.s, on_s.m, on_s.s);
            other->part[x][rank].kl = make_float4(z_ref, t.e, d_here, 0.f);
            mbar_arrive_remote(mapa_u32(&sh.parts[x], uint32_t(lane)));
          }
          __syncwarp();
          wait(&sh.parts[x], (exchanges >> 1) & 1u, 0x603u);
          asm volatile("fence.acq_rel.cluster;" ::: "memory");  // the other CTAs' parts
          ++exchanges;
          float4 p = make_float4(-INFINITY, 0.f, -INFINITY, 0.f), q = make_float4(0.f, 0.f, 0.f, 0.f);
          if (lane < int(ctas)) {
            p = sh.part[x][lane].stats;
            q = sh.part[x][lane].kl;
          }
          st = RowStats{p.x, p.y, 0.f};
          on_s = RowStats{p.z, p.w, 0.f};
          stats_warp<false>(st, a.k);
          if (REST) stats_warp<false>(on_s, a.k);
          z_ref = q.x;
          e_here = q.y;
          d_here = q.z;
        }
        const RowStats rest = REST ? st : stats_empty();
        if (REST) stats_merge(st, on_s, a.k);
        const LkRow w = lk_row<REST>(a, st, rest, t, t_lse, c);
        const float kl = warp_sum(lk_kl(a, w, z_ref, e_here, d_here));  // a CTA's entries in each lane
        if (lane == 0) {
          sh.row[b] = w;
          if (rank == 0) {
            a.kl[r] = w.none ? 0.f : kl + w.rest_kl;
            if (!STEP) a.stats[r] = make_float4(st.m, st.s, rest.m, rest.s);
          }
        }
      }

      // ---- gradient
      if (STEP) {
        named_sync<CT>(2);
        const LkRow& w = sh.row[b];
        if (w.empty || w.none) lk_zero<DT>(in, out, lo, hi, tid, CT);
        else lk_stream_grad<DT, CT>(in, out, lo, hi, w.scale, w.sub, w.off, a.k);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.done[b]);
      __syncwarp();
    }
  }
  __syncthreads();
  if (ctas > 1) cluster_sync();  // no CTA leaves while another may still write to it
}

// Shared memory of a CTA in a cluster of c.
inline int64_t lk_smem(int64_t V, int K, int dtype, int c) {
  const int64_t nv = V / (dtype == KD_F32 ? 4 : 8) + 2;
  return 2 * lk_entry_bytes((nv + c - 1) / c, K);
}

template <int DT, bool REST, bool STEP, int CW, int EW, int PER_SM>
static cudaError_t lk_launch(LogitsKlArgs a, int ctas, cudaStream_t s) {
  static PerDevice<int> ready, resident[LK_MAX_CLUSTER + 1];
  const auto kernel = kd_logits_kl_kernel<DT, REST, STEP, CW, EW, PER_SM>;
  int dev = 0, v = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int rc = ready.get(dev, &v, [&](int, int* out) {
    *out = 1;
    const cudaError_t q = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, LK_MAX_SMEM);
    return int(q != cudaSuccess ? q : cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
  });
  if (rc != 0) return rc > 0 ? cudaError_t(rc) : cudaErrorInvalidDevice;
  const int64_t nv = a.V / Elt<DT>::kVec + 2;
  a.share = int((nv + ctas - 1) / ctas);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(ctas);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3((CW + EW) * 32, 1, 1);
  cfg.dynamicSmemBytes = size_t(lk_smem(a.V, a.K, DT, ctas));
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  int64_t clusters = int64_t(gemm_max_grid()) * PER_SM;
  if (ctas > 1) {
    rc = resident[ctas].get(dev, &v, [&](int, int* out) {
      cudaLaunchConfig_t q = cfg;
      q.gridDim = dim3(unsigned(ctas), 1, 1);
      *out = gemm_max_grid() * PER_SM / ctas;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &q) == cudaSuccess && n >= 1) *out = n;
      return 0;
    });
    if (rc != 0) return rc > 0 ? cudaError_t(rc) : cudaErrorInvalidDevice;
    clusters = v;
  }
  cfg.gridDim = dim3(unsigned((a.N < clusters ? a.N : clusters) * ctas), 1, 1);
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// How a row is shared out, by its bytes (measured: bf16, K = 100, the rest class, N x V; us):
//   up to 16 KB   ten blocks of 4 warps on an SM, a row each: little of a row is its logits
//                 (8192 x 4096: 69; blocks of 5 warps 88, of 9 140)
//   up to 48 KB   eight of 5 warps (4096 x 16000, no rest: 69; of 9 warps some 16 more)
//   up to 96 KB   four of 9 (8192 x 32000, 5 % padding, no rest: 211; of 16 warps some 24 more, of 32
//                 156 more)
//   up to 208 KB  two of 16 (4096 x 100000, no rest: 342; of 9 warps some 28 more, of 32 23 more)
//   longer        one of 32 (2048 x 201088: 339; of 16 warps some 43 more); over 416 KB a cluster of two
//                 or more (1024 x 201088 fp32: 349; without some 20 more), so that the rows in flight
//                 (at most 152 x 4 x 96 KB = 58 MB, 152 x 416 KB = 63 MB) stay in half of L2
// With few rows a cluster takes each, while a thread keeps more than a group of vectors
// (8 x 201088: 22.5; a block each 28.7).
template <int DT, bool REST, bool STEP>
static cudaError_t lk_one(const LogitsKlArgs& a, cudaStream_t s) {
  const int64_t nv = a.V / Elt<DT>::kVec + 2, kb = nv * 16 / 1024;
  const int sms = gemm_max_grid();
  if (kb <= 16) return lk_launch<DT, REST, STEP, 2, 2, 10>(a, 1, s);
  if (kb <= 48 && (a.N > sms || kb <= 32)) return lk_launch<DT, REST, STEP, 4, 1, 8>(a, 1, s);
  if (a.N > sms && kb <= 96) return lk_launch<DT, REST, STEP, 8, 1, 4>(a, 1, s);
  if (a.N > sms && kb <= 208) return lk_launch<DT, REST, STEP, 13, 3, 2>(a, 1, s);
  int c = 1;
  while (c < LK_MAX_CLUSTER && kb > int64_t(416) * c) c *= 2;
  while (2 * c <= LK_MAX_CLUSTER && a.N * c * 2 <= sms && nv >= 2 * c * 1024) c *= 2;
  return lk_launch<DT, REST, STEP, 28, 4, 1>(a, c, s);
}

// ----------------------------------------------------------------- backward ---
// Block (row, slice of the row's vectors).  dz may be z itself: a block reads the logits of its
// entries first and rewrites their gradients last, and every vector is read and written by one
// thread.  One pass over the row: bound by HBM (2 N V elements).  Measured: 300 x 50257 fp32,
// K = 33, the rest class, rows of any alignment: 22.8 us (5.3 TB/s).
template <int DT, bool REST>
__global__ void __launch_bounds__(LKB_THREADS, LKB_PER_SM) kd_logits_kl_bwd_kernel(const LogitsKlArgs a) {
  extern __shared__ __align__(16) uint8_t lkb_raw[];
  __shared__ LkEntryScratch scratch;
  __shared__ LkRow sh_row;
  using raw = typename Elt<DT>::raw;
  constexpr int VE = Elt<DT>::kVec, ET = 128;
  const int64_t r = blockIdx.x / unsigned(a.slices);
  const int slice = int(blockIdx.x % unsigned(a.slices));
  const int tid = int(threadIdx.x);
  const Row<DT> in(static_cast<const raw*>(a.z) + r * a.ld, a.V);
  const Row<DT> out(static_cast<raw*>(a.dz) + r * a.ld_dz, a.V);
  const int share = (in.nv + a.slices - 1) / a.slices;
  const int lo = min(slice * share, in.nv), hi = min(lo + share, in.nv);
  const float4 q = a.stats[r];
  if ((a.mask && a.mask[r] == 0) || q.y == 0.f) {  // padding, or every logit -inf
    lk_zero<DT>(in, out, lo, hi, tid, LKB_THREADS);
    return;
  }
  const LkEntries t = lk_entries(lkb_raw, hi - lo, a.K);
  if (tid < ET) {
    lk_teacher<DT, REST, ET>(a, r, in, lo * VE, hi * VE, t, scratch, lk_ahead<REST>(a, r, tid), tid, slice == 0,
                             [&] { named_sync<ET>(1); }, [&](int id, int) { return in.at(id); });
    if (tid < 32) {
      LkSummary o = lk_nothing();
      if (tid < ET / 32) o = scratch.warp[tid];
      lk_merge(a, o);
      const float n_valid = a.n_valid ? float(*a.n_valid) : float(a.N);
      const LkRow row = lk_row<REST>(a, RowStats{q.x, q.y, 0.f}, RowStats{q.z, q.w, 0.f}, o, scratch.warp[0].t_lse,
                                     *a.grad_loss * a.inv_tau / n_valid);
      if (tid == 0) sh_row = row;
    }
  }
  __syncthreads();
  const LkRow& w = sh_row;
  if (w.none) {  // nothing cached
    lk_zero<DT>(in, out, lo, hi, tid, LKB_THREADS);
    return;
  }
  lk_stream_grad<DT, LKB_THREADS>(in, out, lo, hi, w.scale, w.sub, w.off, a.k);
  __syncthreads();
  lk_write_entries<DT>(a, in, out, lo * VE, t, w, scratch.repeated(ET / 32), tid, LKB_THREADS);
}

template <int DT, bool REST>
static cudaError_t lk_bwd_one(LogitsKlArgs a, cudaStream_t s) {
  static PerDevice<int> done;
  const auto kernel = kd_logits_kl_bwd_kernel<DT, REST>;
  const int64_t nv = a.V / Elt<DT>::kVec + 2;
  // blocks per row: more than one where the rows alone leave SMs idle, while each thread keeps two
  // groups of vectors, or where a row's bitmap is more than a block's share of shared memory
  a.slices = 1;
  while ((a.N * a.slices < int64_t(LKB_PER_SM) * gemm_max_grid() &&
          nv >= int64_t(4) * a.slices * ROW_GROUP * LKB_THREADS) ||
         lk_entry_bytes((nv + a.slices - 1) / a.slices, a.K) > LK_MAX_SMEM)
    a.slices *= 2;
  const int64_t smem = lk_entry_bytes((nv + a.slices - 1) / a.slices, a.K);
  const cudaError_t e = smem_attr_once(done, reinterpret_cast<const void*>(kernel), LK_MAX_SMEM);
  if (e != cudaSuccess) return e;
  kernel<<<unsigned(a.N * a.slices), LKB_THREADS, size_t(smem), s>>>(a);
  return cudaGetLastError();
}

// mode: 1 = forward, 2 = backward, 3 = both in one pass.  Instantiated for each element type in a
// translation unit of its own, which compile at the same time.
template <int DT>
cudaError_t lk_run(int mode, const LogitsKlArgs& a, cudaStream_t s) {
  const bool rest = a.t_lse != nullptr;
  if (mode == 1) return rest ? lk_one<DT, true, false>(a, s) : lk_one<DT, false, false>(a, s);
  if (mode == 2) return rest ? lk_bwd_one<DT, true>(a, s) : lk_bwd_one<DT, false>(a, s);
  return rest ? lk_one<DT, true, true>(a, s) : lk_one<DT, false, true>(a, s);
}

}  // namespace kd
