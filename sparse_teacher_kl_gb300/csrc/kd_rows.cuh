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
template <int DT>
__device__ __forceinline__ float group_max(const uint4 (&v)[ROW_GROUP]) {
  if constexpr (DT == KD_F32) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < ROW_GROUP; ++j) {
      const float a = max_nan(__uint_as_float(v[j].x), __uint_as_float(v[j].y));
      const float b = max_nan(__uint_as_float(v[j].z), __uint_as_float(v[j].w));
      m = max_nan(m, max_nan(a, b));
    }
    return m;
  } else {
    uint32_t m = Elt<DT>::kNegInf;
#pragma unroll
    for (int j = 0; j < ROW_GROUP; ++j)
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
  // The vectors first, first + step, ... (ROW_GROUP of them) below `end`; -inf from there on.
  __device__ __forceinline__ void load_group(uint4 (&v)[ROW_GROUP], int first, int step, int end) const {
    if (first >= full_lo && int64_t(first) + int64_t(ROW_GROUP - 1) * step < (end < full_hi ? end : full_hi)) {
#pragma unroll
      for (int j = 0; j < ROW_GROUP; ++j) v[j] = __ldcs(reinterpret_cast<const uint4*>(base) + first + j * step);
    } else {
#pragma unroll
      for (int j = 0; j < ROW_GROUP; ++j) {
        const int64_t i = int64_t(first) + int64_t(j) * step;
        v[j] = i < end ? load(int(i))
                       : make_uint4(Elt<DT>::kNegInf, Elt<DT>::kNegInf, Elt<DT>::kNegInf, Elt<DT>::kNegInf);
      }
    }
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
// Over the elements x seen so far, with k = log2(e) / tau:
//   m = max x,  s = sum 2^((x - m) k),  u = sum 2^((x - m) k) (x - m) k
// so that logsumexp(x / tau) = m / tau + ln s and the entropy of softmax(x / tau) is
// ln s - ln2 u / s: a sum of two terms that are never negative.  x - m is formed first
// (exact for neighbours, and finite or -inf even for masks of a type's lowest value), then
// scaled.  An empty set has m = -inf, s = 0; a NaN makes s NaN (m skips it).

struct RowStats {
  float m = -INFINITY, s = 0.f, u = 0.f;
};

// 2^t of a difference of maxima; t = -inf (one side empty or far below) gives 0.
__device__ __forceinline__ float stats_shift(float from, float to, float k, float& t) {
  t = fmaxf((from - to) * k, -200.f);  // 2^-200 is 0 in fp32; keeps t * 0 finite
  return ex2_approx(t);
}

__device__ __forceinline__ void stats_merge(RowStats& a, const RowStats& b, float k) {
  const float M = fmaxf(a.m, b.m);
  if (M == -INFINITY) {
    a.s += b.s;  // 0, or NaN where a side held one
    return;
  }
  float ta = 0.f, tb = 0.f;
  const float fa = a.m == M ? 1.f : (a.m == -INFINITY ? 0.f : stats_shift(a.m, M, k, ta));
  const float fb = b.m == M ? 1.f : (b.m == -INFINITY ? 0.f : stats_shift(b.m, M, k, tb));
  const float u = fmaf(ta, a.s, a.u) * fa + fmaf(tb, b.s, b.u) * fb;
  a.s = a.s * fa + b.s * fb;
  a.u = u;
  a.m = M;
}

// Add the elements of a thread's vectors, whose largest is gmax.
template <int DT, bool ENT>
__device__ __forceinline__ void stats_add(RowStats& st, const uint4 (&v)[ROW_GROUP], float gmax, float k) {
  if (gmax == -INFINITY) return;
  if (!(gmax <= st.m)) {
    if (gmax != gmax) {
      st.s = gmax;
      return;
    }
    if (st.m != -INFINITY) {
      float t;
      const float f = stats_shift(st.m, gmax, k, t);
      if (ENT) st.u = fmaf(t, st.s, st.u) * f;
      st.s *= f;
    }
    st.m = gmax;
  }
#pragma unroll
  for (int j = 0; j < ROW_GROUP; ++j) {
    float x[Elt<DT>::kVec];
    unpack_vec<DT>(v[j], x);
#pragma unroll
    for (int e = 0; e < Elt<DT>::kVec; ++e) {
      const float t = (x[e] - st.m) * k;
      const float p = ex2_approx(t);
      st.s += p;
      if (ENT) st.u = fmaf(p, fmaxf(t, -200.f), st.u);
    }
  }
}

__device__ __forceinline__ RowStats stats_shfl_xor(const RowStats& a, int o) {
  RowStats b;
  b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
  b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
  b.u = __shfl_xor_sync(0xffffffffu, a.u, o);
  return b;
}

// The block's statistics in every thread; `sh`: one entry per warp.
template <int THREADS>
__device__ __forceinline__ RowStats stats_block(RowStats st, float k, RowStats* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) stats_merge(st, stats_shfl_xor(st, o), k);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) sh[warp] = st;
  __syncthreads();
  st = lane < THREADS / 32 ? sh[lane] : RowStats{};
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) stats_merge(st, stats_shfl_xor(st, o), k);
  // a merge rounds differently from its mirror image: every thread takes lane 0's result
  st.m = __shfl_sync(0xffffffffu, st.m, 0);
  st.s = __shfl_sync(0xffffffffu, st.s, 0);
  st.u = __shfl_sync(0xffffffffu, st.u, 0);
  return st;
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

// Call f.template operator()<DT>() for a run-time element type.
#define KD_DISPATCH_TYPE(dt, ...)                                             \
  do {                                                                        \
    if ((dt) == KD_BF16) { constexpr int DT = KD_BF16; __VA_ARGS__; }         \
    else if ((dt) == KD_F16) { constexpr int DT = KD_F16; __VA_ARGS__; }      \
    else { constexpr int DT = KD_F32; __VA_ARGS__; }                          \
  } while (0)

}  // namespace kd
