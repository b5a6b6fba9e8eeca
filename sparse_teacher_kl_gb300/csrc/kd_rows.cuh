// Reading and writing dense logit rows: element types, 16-byte vectors over rows of any
// alignment, and the running statistics of a softmax.
//
// A row of V elements is covered by a grid of 16-byte vectors laid from the last 16-byte
// boundary at or before its first element, so that every vector inside the row is one aligned
// access whatever the row's stride.  The (at most two) vectors that the row only partly covers
// are read and written element by element; nothing outside the row is touched.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "kd_device.cuh"
#include "kd_internal.h"

namespace kd {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int ROW_GROUP = 4;  // vectors that a thread has in flight

// ------------------------------------------------------------- elements ---

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <int DT>
struct Elt;  // DT: KD_BF16, KD_F16, KD_F32

template <>
struct Elt<KD_BF16> {
  using raw = uint16_t;
  static constexpr int kVec = 8;
  static constexpr uint32_t kNegInf = 0xFF80FF80u;  // one word of -inf elements
  static __device__ __forceinline__ float widen(raw r) { return __uint_as_float(uint32_t(r) << 16); }
  static __device__ __forceinline__ void unpack(uint32_t w, float& a, float& b) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xFFFF0000u);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) { return pack_bf16x2(a, b); }
  static __device__ __forceinline__ raw narrow(float a) { return raw(pack_bf16x2(a, a) & 0xFFFFu); }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};

template <>
struct Elt<KD_F16> {
  using raw = uint16_t;
  static constexpr int kVec = 8;
  static constexpr uint32_t kNegInf = 0xFC00FC00u;
  static __device__ __forceinline__ float widen(raw r) { return __half2float(__ushort_as_half(r)); }
  static __device__ __forceinline__ void unpack(uint32_t w, float& a, float& b) {
    a = __half2float(__ushort_as_half(uint16_t(w & 0xFFFFu)));
    b = __half2float(__ushort_as_half(uint16_t(w >> 16)));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
  }
  static __device__ __forceinline__ raw narrow(float a) { return raw(pack(a, a) & 0xFFFFu); }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};

template <>
struct Elt<KD_F32> {
  using raw = uint32_t;
  static constexpr int kVec = 4;
  static constexpr uint32_t kNegInf = 0xFF800000u;
  static __device__ __forceinline__ float widen(raw r) { return __uint_as_float(r); }
  static __device__ __forceinline__ raw narrow(float a) { return __float_as_uint(a); }
};

// The elements of a vector as floats, and back (one rounding to nearest).
template <int DT>
__device__ __forceinline__ void unpack_vec(const uint4& v, float (&x)[Elt<DT>::kVec]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    if constexpr (DT == KD_F32) x[h] = __uint_as_float(w[h]);
    else Elt<DT>::unpack(w[h], x[2 * h], x[2 * h + 1]);
  }
}

template <int DT>
__device__ __forceinline__ uint4 pack_vec(const float (&x)[Elt<DT>::kVec]) {
  if constexpr (DT == KD_F32)
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  else
    return make_uint4(Elt<DT>::pack(x[0], x[1]), Elt<DT>::pack(x[2], x[3]), Elt<DT>::pack(x[4], x[5]),
                      Elt<DT>::pack(x[6], x[7]));
}

// Largest element of a thread's vectors; NaN if one of them is NaN.
template <int DT, int N>
__device__ __forceinline__ float group_max(const uint4 (&v)[N]) {
  if constexpr (DT == KD_F32) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float a = max_nan(__uint_as_float(v[j].x), __uint_as_float(v[j].y));
      const float b = max_nan(__uint_as_float(v[j].z), __uint_as_float(v[j].w));
      m = max_nan(m, max_nan(a, b));
    }
    return m;
  } else {
    uint32_t m = Elt<DT>::kNegInf;
#pragma unroll
    for (int j = 0; j < N; ++j)
      m = Elt<DT>::max2(m, Elt<DT>::max2(Elt<DT>::max2(v[j].x, v[j].y), Elt<DT>::max2(v[j].z, v[j].w)));
    float a, b;
    Elt<DT>::unpack(m, a, b);
    return max_nan(a, b);
  }
}

// ----------------------------------------------------------------- rows ---

template <int DT>
struct Row {
  using raw = typename Elt<DT>::raw;
  static constexpr int kVec = Elt<DT>::kVec;
  uint8_t* base;   // the 16-byte boundary of vector 0
  int lead;        // elements of vector 0 that lie before the row
  int V;           // elements
  int nv;          // vectors
  int full_lo, full_hi;  // vectors [full_lo, full_hi) lie wholly inside the row

  __device__ __forceinline__ Row(const void* p, int V_) : V(V_) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    lead = int((at & 15u) / sizeof(raw));
    base = reinterpret_cast<uint8_t*>(at & ~uintptr_t(15));
    nv = int((int64_t(lead) + V + kVec - 1) / kVec);
    full_lo = lead ? 1 : 0;
    full_hi = int((int64_t(lead) + V) / kVec);
  }
  __device__ __forceinline__ raw* elt(int64_t col) const { return reinterpret_cast<raw*>(base) + lead + col; }
  __device__ __forceinline__ float at(int64_t col) const { return Elt<DT>::widen(*elt(col)); }
  __device__ __forceinline__ bool whole(int i) const { return i >= full_lo && i < full_hi; }
  __device__ __forceinline__ int64_t col(int i) const { return int64_t(i) * kVec - lead; }  // of vector i's element 0

  // Vector i; the elements outside the row are -inf.
  __device__ __forceinline__ uint4 load_edge(int i) const {
    uint32_t w[4] = {Elt<DT>::kNegInf, Elt<DT>::kNegInf, Elt<DT>::kNegInf, Elt<DT>::kNegInf};
    const int64_t c0 = col(i);
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      if (c0 + e >= 0 && c0 + e < V) {
        const uint32_t r = *elt(c0 + e);
        if constexpr (DT == KD_F32) w[e] = r;
        else w[e >> 1] = (e & 1) ? ((w[e >> 1] & 0xFFFFu) | (r << 16)) : ((w[e >> 1] & 0xFFFF0000u) | r);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ uint4 load(int i) const {
    if (whole(i)) return __ldcs(reinterpret_cast<const uint4*>(base) + i);
    return load_edge(i);
  }
  // Elements of vector i of a row that starts `lead_` elements into its grid, written to this row.
  __device__ __forceinline__ void store(int i, int lead_, const float (&x)[kVec]) const {
    if (lead_ == lead && whole(i)) {
      __stcs(reinterpret_cast<uint4*>(base) + i, pack_vec<DT>(x));
      return;
    }
    const int64_t c0 = int64_t(i) * kVec - lead_;
#pragma unroll
    for (int e = 0; e < kVec; ++e)
      if (c0 + e >= 0 && c0 + e < V) *elt(c0 + e) = Elt<DT>::narrow(x[e]);
  }
};

// ----------------------------------------------------- softmax statistics ---
// Over the elements x seen so far, with k = log2(e) / tau and t(x) = x k - O(m):
//   m = max x,  s = sum 2^t,  u = sum 2^t t
// so that log2 of p(x) is t(x) - log2 s, logsumexp(x / tau) is ln2 (O(m) + log2 s) and the
// entropy of softmax(x / tau) is ln2 (log2 s - u / s).  The offset O(m) is
//   fl(m k)  where |m k| is up to 2^20: t is one fused multiply-add against the same rounded
//            offset everywhere, so its rounding (up to 2^-5) cancels;
//   m k      elsewhere (small temperatures, masks of large finite values), unrounded: there the
//            rounding would reach 2^7 and more and the sums overflow, so t is (x - m) k.
// An empty set has m = -inf, s = 0; a NaN or +inf element makes s NaN (m skips a NaN).

struct RowStats {
  float m, s, u;
};
__device__ __forceinline__ RowStats stats_empty() { return {-INFINITY, 0.f, 0.f}; }

constexpr float kPlainMax = 1048576.f;  // of |m k|

// Whether the offset of maximum m is rounded; its rounding, m k - O(m).
__device__ __forceinline__ bool stats_plain(float m, float k) { return fabsf(__fmul_rn(m, k)) <= kPlainMax; }
__device__ __forceinline__ float stats_rounding(float m, float k) {
  const float o = __fmul_rn(m, k);
  return fabsf(o) <= kPlainMax ? fmaf(m, k, -o) : 0.f;
}

__device__ __forceinline__ float stats_t(float x, float m, float k) {
  const float o = __fmul_rn(m, k);
  return fabsf(o) <= kPlainMax ? fmaf(x, k, -o) : (x - m) * k;
}

// ln p of an element from its row's statistics, log2_s = log2 of s.  Where x k would overflow
// although the log probability need not, x / tau is formed instead (fl(m k)'s rounding is nothing
// beside it).
__device__ __forceinline__ float stats_logp(float x, float m, float log2_s, float k, float tau) {
  if (stats_plain(m, k) && fabsf(__fmul_rn(x, k)) <= 1e30f) return kLn2 * (stats_t(x, m, k) - log2_s);
  return (x - m) / tau - kLn2 * log2_s;
}

// logsumexp(x / tau); infinite where fp32 does not hold it.
__device__ __forceinline__ float stats_lse(float m, float log2_s, float k, float tau) {
  return stats_plain(m, k) ? kLn2 * (__fmul_rn(m, k) + log2_s) : m / tau + kLn2 * log2_s;
}

// log2 of the factor that takes a sum relative to `from` to one relative to `to`: O(from) - O(to).
// The unlikely half is a call, so that it takes no registers of the loops around it (scoring 4096 x
// 151936: 217 us; in line 227).
static __device__ __noinline__ float stats_shift_far(float from, float to, float k) {
  return (from - to) * k + (stats_rounding(to, k) - stats_rounding(from, k));
}
__device__ __forceinline__ float stats_shift(float from, float to, float k) {
  const float a = __fmul_rn(from, k), b = __fmul_rn(to, k);
  return fmaxf(fabsf(a), fabsf(b)) <= kPlainMax ? a - b : stats_shift_far(from, to, k);
}

__device__ __forceinline__ void stats_rescale(RowStats& a, float to, float k) {
  if (a.m == to || a.m == -INFINITY) {  // nothing summed yet: s is 0, or NaN
    a.m = to;
    return;
  }
  // -200 stands for anything that far below (2^-200 is 0 in fp32, and -200 times 0 is 0)
  const float t = fmaxf(stats_shift(a.m, to, k), -200.f), f = ex2_approx(t);
  a.u = fmaf(t, a.s, a.u) * f;
  a.s *= f;
  a.m = to;
}

__device__ __forceinline__ void stats_merge(RowStats& a, RowStats b, float k) {
  const float M = fmaxf(a.m, b.m);
  if (M != -INFINITY) {
    stats_rescale(a, M, k);
    stats_rescale(b, M, k);
  }
  a.s += b.s;
  a.u += b.u;
}

// Two floats in one 64-bit register, for the packed fp32 instructions.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Add the elements of N vectors whose largest element is gmax.
template <int DT, bool ENT, int N>
__device__ __forceinline__ void stats_add(RowStats& st, const uint4 (&v)[N], float gmax, float k) {
  constexpr int VE = Elt<DT>::kVec;
  if (gmax == -INFINITY) return;
  if (!(gmax <= st.m)) {
    if (gmax != gmax) {
      st.s = gmax;
      return;
    }
    stats_rescale(st, gmax, k);
  }
  // An element of -inf has weight 0, but its exponent must stay finite for u: elements are
  // raised to a floor, which changes nothing while the floor's own weight is 0 and its exponent
  // finite (not at temperatures below 1e-8, nor fp16 ones above a few hundred: the loop below then).
  constexpr float kFloor = DT == KD_F16 ? -65504.f : -1e30f;
  const float off = -__fmul_rn(st.m, k), low = (st.m - kFloor) * k;
  if (fabsf(off) <= kPlainMax && (!ENT || (low > 150.f && low < 1e38f))) {
    const uint64_t k2 = pack2(k, k), off2 = pack2(off, off);
    uint64_t s2[2] = {0, 0}, u2[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
      for (int h = 0; h < VE / 2; ++h) {
        float x0, x1;
        if constexpr (DT == KD_F32) {
          x0 = __uint_as_float(w[2 * h]);
          x1 = __uint_as_float(w[2 * h + 1]);
          if (ENT) {
            x0 = max_nan(x0, kFloor);
            x1 = max_nan(x1, kFloor);
          }
        } else {
          constexpr uint32_t low = DT == KD_F16 ? 0xFBFFFBFFu : 0xF14AF14Au;  // -65504; -1e30 in bf16
          Elt<DT>::unpack(ENT ? Elt<DT>::max2(w[h], low) : w[h], x0, x1);
        }
        const uint64_t t2 = fma2(pack2(x0, x1), k2, off2);
        float t0, t1;
        unpack2(t2, t0, t1);
        const uint64_t p2 = pack2(ex2_approx(t0), ex2_approx(t1));
        s2[h & 1] = add2(s2[h & 1], p2);
        if (ENT) u2[h & 1] = fma2(p2, t2, u2[h & 1]);
      }
    }
    float a, b;
    unpack2(add2(s2[0], s2[1]), a, b);
    st.s += a + b;
    if (ENT) {
      unpack2(add2(u2[0], u2[1]), a, b);
      st.u += a + b;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    float x[VE];
    unpack_vec<DT>(v[j], x);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const float t = stats_t(x[e], st.m, k), p = ex2_approx(t);
      st.s += p;
      if (ENT) st.u = fmaf(p, fmaxf(t, -200.f), st.u);
    }
  }
}

__device__ __forceinline__ float warp_max(float x, int width = 32) {
  for (int o = width / 2; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x, int width = 32) {
  for (int o = width / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The statistics of `width` consecutive lanes (a power of two), in each of them.
template <bool ENT>
__device__ __forceinline__ void stats_warp(RowStats& st, float k, int width = 32) {
  const float M = warp_max(st.m, width);
  if (M != -INFINITY) stats_rescale(st, M, k);
  st.s = warp_sum(st.s, width);
  if (ENT) st.u = warp_sum(st.u, width);
}

// The block's statistics in every thread, in two halves with a barrier of the caller's between
// them.  `sh`: one entry per warp.
template <bool ENT>
__device__ __forceinline__ void stats_block_put(RowStats st, float k, RowStats* sh) {
  stats_warp<ENT>(st, k);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = st;
}
template <int THREADS, bool ENT>
__device__ __forceinline__ RowStats stats_block_get(float k, const RowStats* sh) {
  constexpr int W = THREADS / 32;
  RowStats st = sh[threadIdx.x & (W - 1)];
  stats_warp<ENT>(st, k, W);
  return st;
}
template <int THREADS, bool ENT>
__device__ __forceinline__ RowStats stats_block(const RowStats& st, float k, RowStats* sh) {
  stats_block_put<ENT>(st, k, sh);
  __syncthreads();
  return stats_block_get<THREADS, ENT>(k, sh);
}

// Loads of a row that is read once, and of one that is read again soon: the second asks L2 to keep
// the lines.
struct LoadOnce {
  __device__ __forceinline__ uint4 operator()(const uint4* p) const { return __ldcs(p); }
};
struct LoadKeep {
  uint64_t policy;
  __device__ __forceinline__ LoadKeep() {
    asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(policy));
  }
  __device__ __forceinline__ uint4 operator()(const uint4* p) const {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p), "l"(policy));
    return v;
  }
};

// Stream vectors [lo, hi) of a row through the block's first THREADS threads, ROW_GROUP vectors of a
// thread at a time:
//   get(address)         reads a vector
//   fix(vector, i)       may change vector i before it is added
//   on_group(round, max) sees the largest element of each group of a thread
// The vectors that the row only partly covers are added last, one thread each.
template <int DT, bool ENT, int THREADS, class Load, class Fix, class OnGroup>
__device__ __forceinline__ void stream_stats(const Row<DT>& row, int lo, int hi, float k, RowStats& st, Load&& get,
                                             Fix&& fix, OnGroup&& on_group) {
  constexpr uint32_t NI = Elt<DT>::kNegInf;
  const int first = max(lo, row.full_lo) + int(threadIdx.x), end = min(hi, row.full_hi);
  const uint4* p = reinterpret_cast<const uint4*>(row.base);
  constexpr int STEP = ROW_GROUP * THREADS;
  auto load = [&](uint4 (&v)[ROW_GROUP], int i0) {
    if (i0 + (ROW_GROUP - 1) * THREADS < end) {
#pragma unroll
      for (int j = 0; j < ROW_GROUP; ++j) v[j] = get(p + i0 + j * THREADS);
    } else {
#pragma unroll
      for (int j = 0; j < ROW_GROUP; ++j)
        v[j] = i0 + j * THREADS < end ? get(p + i0 + j * THREADS) : make_uint4(NI, NI, NI, NI);
    }
  };
  int round = 0, i0 = first;
  auto add = [&](uint4 (&v)[ROW_GROUP]) {
#pragma unroll
    for (int j = 0; j < ROW_GROUP; ++j) fix(v[j], i0 + j * THREADS);
    const float g = group_max<DT>(v);
    on_group(round, g);
    stats_add<DT, ENT>(st, v, g, k);
    i0 += STEP;
    ++round;
  };
  // one set of registers: a second one, loaded while the first is added, measured slower, since it
  // halves the warps that an SM holds
  while (i0 < end) {
    uint4 v[ROW_GROUP];
    load(v, i0);
    add(v);
  }
  const int edge = threadIdx.x == 0 ? 0 : row.nv - 1;
  if (threadIdx.x < 2 && edge >= lo && edge < hi && !row.whole(edge) && (threadIdx.x == 0 || edge != 0)) {
    uint4 v[1] = {row.load_edge(edge)};
    fix(v[0], edge);
    stats_add<DT, ENT>(st, v, group_max<DT>(v), k);
  }
}

template <int THREADS>
__device__ __forceinline__ float sum_block(float x, float* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) sh[warp] = x;
  __syncthreads();
  x = lane < THREADS / 32 ? sh[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Order-preserving 32-bit key of a float; the zeros are equal.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

// Map vectors [lo, hi) of a row through the block's first THREADS threads: x = f(x) for every
// element, from `in` to `out` (in place where they are the same row).  Whole vectors of rows that
// are aligned alike go as such, ROW_GROUP of a thread at a time; the others by elements.
template <int DT, int THREADS, class F>
__device__ __forceinline__ void stream_map(const Row<DT>& in, const Row<DT>& out, int lo, int hi, F&& f) {
  constexpr int VE = Elt<DT>::kVec, STEP = ROW_GROUP * THREADS;
  const bool alike = in.lead == out.lead;
  const int body_lo = max(lo, in.full_lo), body_hi = max(body_lo, min(hi, in.full_hi));
  if (alike) {
    const uint4* p = reinterpret_cast<const uint4*>(in.base) + body_lo + threadIdx.x;
    uint4* o = reinterpret_cast<uint4*>(out.base) + body_lo + threadIdx.x;
    int left = body_hi - body_lo - int(threadIdx.x);  // vectors from this one on
    for (; left > (ROW_GROUP - 1) * THREADS; left -= STEP, p += STEP, o += STEP) {
      uint4 v[ROW_GROUP];
#pragma unroll
      for (int j = 0; j < ROW_GROUP; ++j) v[j] = __ldcs(p + j * THREADS);
#pragma unroll
      for (int j = 0; j < ROW_GROUP; ++j) {
        float x[VE];
        unpack_vec<DT>(v[j], x);
        f(x);
        __stcs(o + j * THREADS, pack_vec<DT>(x));
      }
    }
    for (; left > 0; left -= THREADS, p += THREADS, o += THREADS) {
      float x[VE];
      unpack_vec<DT>(__ldcs(p), x);
      f(x);
      __stcs(o, pack_vec<DT>(x));
    }
  } else {
    for (int i = body_lo + int(threadIdx.x); i < body_hi; i += THREADS) {
      float x[VE];
      unpack_vec<DT>(in.load(i), x);
      f(x);
      out.store(i, in.lead, x);
    }
  }
  const int edge = threadIdx.x == 0 ? 0 : in.nv - 1;
  if (threadIdx.x < 2 && edge >= lo && edge < hi && !in.whole(edge) && (threadIdx.x == 0 || edge != 0)) {
    float x[VE];
    unpack_vec<DT>(in.load_edge(edge), x);
    f(x);
    out.store(edge, in.lead, x);
  }
}

// Call f.template operator()<DT>() for a run-time element type.
#define KD_DISPATCH_TYPE(dt, ...)                                             \
  do {                                                                        \
    if ((dt) == KD_BF16) { constexpr int DT = KD_BF16; __VA_ARGS__; }         \
    else if ((dt) == KD_F16) { constexpr int DT = KD_F16; __VA_ARGS__; }      \
    else { constexpr int DT = KD_F32; __VA_ARGS__; }                          \
  } while (0)

}  // namespace kd
