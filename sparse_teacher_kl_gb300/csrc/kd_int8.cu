// 8-bit integers: rows quantised with one scale each, and the product of two such matrices,
//   quantize   s_n = max_k |x_nk| / 127,  q_nk = x_nk / s_n to the nearest whole number (ties to even)
//   product    C_mn = (sum_k A_mk B_nk) sa_m sb_n
// A: [M, K], the tokens; B: [N, K], the channels (a head's vocabulary, a layer's outputs).
//
// sm_103a's fast tensor path takes no 8-bit integers, but every one of them is a 16-bit floating-point
// number, and so is their product a sum of exact terms: fp16 operands and fp32 accumulators give the integer
// sums themselves as long as those stay within 2^24 (always for K <= 1024; at K = 4096 a standard deviation of the
// sum of uniform integers is 2^24 / 48, and the largest of 5 million sums 2^24 / 9; normal rows scaled by their
// largest stay 40 times away), and beyond that sums that each step of 16 cuts off to fp32.  So the operations cannot go
// faster than the 16-bit rate, but the weights keep their single byte all the way from HBM to the SM:
// they are widened on their way from shared to tensor memory, where tcgen05.mma takes its A operand from.
//
// Measured, K = 2880, N = 201088, bf16 out (us; TB/s of what must move, or PFLOP/s): 1 token 92 (6.2 TB/s, 93 % of the
// copy), 5 98 (5.9), 64 109 (5.5), 128 118, 256 180 (1.65 PFLOP/s), 512 325 (1.82), 4096 2690 (1.76 in a row, 1.95 alone,
// 91 % and 101 % of the bf16 rate); quantising 8192 x 4096 bf16 26 us (3.9 TB/s), fp32 29 (5.8), 1 x 2880 2.6.
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "kd_device.cuh"
#include "kd_internal.h"

namespace kd {

namespace {

// ------------------------------------------------------------------ geometry ---
// A tile is 128 channels (the MMA's M side, from tensor memory) by TN tokens (its N side, from shared
// memory); a pair of CTAs computes 256 channels, each loading half of the tokens.  The reduction goes 128
// deep a stage.  Tensor memory's 512 columns: four stages of widened weights, which cover the way from an
// MMA's end over the barriers to the next weights' arrival (about 1300 cycles; two stages left the tensor
// cores waiting a third of the time), and one accumulator of up to 256 tokens, or two of up to 128.  One large
// accumulator, whose draining the next tile waits for, beats two of 192 (4096 x 2880 x 201088 3.5 ms against 3.95,
// before the later steps): an MMA takes 40 to 60 cycles to issue, and short ones (96 cycles for 192 tokens)
// leave the issuing warp little for its barriers.
constexpr int T8_ROWS = 128;
constexpr int T8_K = 128;
constexpr int T8_W_BYTES = T8_ROWS * T8_K;      // a stage's weights: 16 KB
constexpr int T8_MAX_TOKENS = 256;
constexpr int T8_TWO_ACC = 128;                 // tokens up to which there are two accumulators
constexpr int T8_SHORT_K = 768;                 // K up to which no tile has more
// Shared memory: two rings of stages, since a stage's weights are free as soon as they have been widened and its
// tokens only when its MMAs are done: these go round with the widened weights, on one barrier.
constexpr int T8_MAX_STAGES = 8;
constexpr int T8_WIDE = 4;                      // stages of widened weights, 64 columns each
constexpr int T8_ACC_COL = T8_WIDE * 64;
// Sets of 4 widening warps, taking stages in turn (three or four leave the epilogue's and the MMA warp too few of
// the schedulers' slots: 4096 x 2880 x 201088 2.69 ms with two, 2.73 and 2.94; 2000 x 256 x 100000 185 us, 299 and
// 285).  The ring of weights is a multiple of the sets long, so that a place in it is always the same set's: a wait
// by parity is only right for who has seen the barrier's last phase, and loads may land out of order.
constexpr int T8_SETS = 2;
static_assert(T8_MAX_STAGES % T8_SETS == 0, "places of the weights' ring belong to a set");
constexpr int T8_EPI = 8;                       // epilogue warps, two to a quarter of the lanes
// Warps: weights' and tokens' TMA (0, 2), MMA (1), none (3), epilogue, widening.
constexpr int T8_THREADS = 32 * (4 + T8_EPI + 4 * T8_SETS);
constexpr int T8_SMEM = 227 * 1024;

struct __align__(16) T8Tail {
  uint64_t wgot[T8_MAX_STAGES], wempty[T8_MAX_STAGES];  // weights
  uint64_t tgot[T8_WIDE];                               // tokens; free with the weights widened for them
  uint64_t wide[T8_WIDE], wfree[T8_WIDE];
  uint64_t tfull[2], tempty[2];
  uint64_t drain;
  uint32_t tmem_base, abort_flag;
  float a_scale[T8_EPI][128];  // of each epilogue warp's tokens
};

static_assert((T8_SMEM - 1024 - int(sizeof(T8Tail)) - T8_WIDE * (T8_MAX_TOKENS / 2 * 256)) / T8_W_BYTES >= T8_SETS,
              "a place for every set beside the largest tiles' tokens");

struct T8Problem {
  int M, N, K;
  int tokens;        // TN: tokens of a tile, a multiple of 16 (a pair's: of 32)
  int token_tiles, units, w_stages, t_bytes;
  const float *a_scale, *b_scale;
  void* C;
  int64_t ldc;
  uint32_t* err;
};

// Four integers to two pairs of fp16: with the sign bit flipped a byte is x + 128, the low mantissa bits of
// 1024 + that; 1152 taken away again is exact.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));
  uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), bias), y = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void store_out(uint16_t* p, float v) { *p = uint16_t(pack_bf16x2(v, v)); }

// A place in a ring of `n` stages and the parity of its turn; by steps of at most n.
struct Turn {
  uint32_t at, parity;
  __device__ __forceinline__ void step(uint32_t by, uint32_t n) {
    at += by;
    if (at >= n) {
      at -= n;
      parity ^= 1u;
    }
  }
};

// A CTA's (pair's) units in turn: unit u is channel group u / token_tiles, token tile u % token_tiles.
struct Walk {
  int u, group, tile;
  __device__ __forceinline__ Walk(const T8Problem& p, int first) : u(first), group(first / p.token_tiles) {
    tile = first - group * p.token_tiles;
  }
  __device__ __forceinline__ void step(const T8Problem& p, int by, int by_groups, int by_tiles) {
    u += by;
    group += by_groups;
    tile += by_tiles;
    if (tile >= p.token_tiles) {
      tile -= p.token_tiles;
      ++group;
    }
  }
};

template <class OUT>
__device__ __forceinline__ uint32_t pack_out(float lo, float hi) {
  return pack_bf16x2(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t pack_out<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two tokens' values of a channel.
template <class OUT>
__device__ __forceinline__ void store_pair(OUT* a, OUT* b, float x, float y) {
  if constexpr (sizeof(OUT) == 4) {
    *a = x;
    *b = y;
  } else {
    const uint32_t w = pack_out<OUT>(x, y);
    *reinterpret_cast<uint16_t*>(a) = uint16_t(w & 0xFFFFu);
    *reinterpret_cast<uint16_t*>(b) = uint16_t(w >> 16);
  }
}

template <int CG, class OUT>
__global__ void __launch_bounds__(T8_THREADS, 1)
    kd_gemm8_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_t,
                    const T8Problem p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* smem_t = smem + size_t(p.w_stages) * T8_W_BYTES;
  T8Tail* tail = reinterpret_cast<T8Tail*>(smem_t + size_t(T8_WIDE) * p.t_bytes);
  const uint32_t w_stages = uint32_t(p.w_stages);
  volatile uint32_t* abort_flag = &tail->abort_flag;
  const uint32_t warp = threadIdx.x >> 5, lane = lane_id();
  const uint32_t crank = CG == 2 ? cluster_ctarank() : 0u;
  const int u_first = int(blockIdx.x) / CG, u_step = int(gridDim.x) / CG;
  const int k_stages = (p.K + T8_K - 1) / T8_K;
  const int step_groups = u_step / p.token_tiles, step_tiles = u_step - step_groups * p.token_tiles;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.w_stages; ++s) {
      mbar_init(&tail->wgot[s], 1);
      mbar_init(&tail->wempty[s], 4);  // a lane of each warp of the set that widened them
    }
    for (int t = 0; t < T8_WIDE; ++t) {
      mbar_init(&tail->tgot[t], 1);
      mbar_init(&tail->wide[t], 4 * CG);  // a lane of each widening warp, of both CTAs
      mbar_init(&tail->wfree[t], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tail->tfull[a], 1);
      mbar_init(&tail->tempty[a], T8_EPI * CG);
    }
    mbar_init(&tail->drain, 1);
    tail->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&tmap_w);
    tma_prefetch_map(&tmap_t);
  }
  if (warp == 1) {
    if (CG == 2) tmem_alloc_pair(&tail->tmem_base, TMEM_COLS); else tmem_alloc(&tail->tmem_base, TMEM_COLS);
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();  // the peer's barriers exist before any commit reaches them
  tc_fence_after();
  const uint32_t tmem_base = tail->tmem_base;
  const uint32_t accs = p.tokens <= T8_TWO_ACC ? 2u : 1u;

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ TMA producers
    if (lane == 0) {
      const bool tokens = warp == 2;
      const uint32_t stages = tokens ? uint32_t(T8_WIDE) : w_stages;
      uint64_t* got = tokens ? tail->tgot : tail->wgot;
      uint64_t* empty = tokens ? tail->wfree : tail->wempty;
      const int rows_t = p.tokens / CG;
      uint32_t it = 0;
      Turn r{0, 0};
      bool ok = true;
      for (Walk at(p, u_first); at.u < p.units && ok; at.step(p, u_step, step_groups, step_tiles)) {
        const int row = (at.group * CG + int(crank)) * T8_ROWS, tok = at.tile * p.tokens + int(crank) * rows_t;
        for (int kb = 0; kb < k_stages; ++kb, ++it, r.step(1, stages)) {
          if (!mbar_wait_suspended(&empty[r.at], r.parity ^ 1u, abort_flag, p.err, 0x1100u + warp)) {
            ok = false;
            break;
          }
          if (tokens && CG == 2) {
            // both CTAs' halves complete on the first CTA's barrier, where the MMAs wait
            if (crank == 0) mbar_arrive_expect_tx(&got[r.at], 2u * uint32_t(p.t_bytes));
            tma_load_3d_pair(smem_t + size_t(r.at) * p.t_bytes, &tmap_t, mapa_u32(&got[r.at], 0), 0, tok, kb * 2);
          } else if (tokens) {
            mbar_arrive_expect_tx(&got[r.at], uint32_t(p.t_bytes));
            tma_load_3d(smem_t + size_t(r.at) * p.t_bytes, &tmap_t, &got[r.at], 0, tok, kb * 2);
          } else {
            mbar_arrive_expect_tx(&got[r.at], uint32_t(T8_W_BYTES));
            tma_load_2d(smem + size_t(r.at) * T8_W_BYTES, &tmap_w, &got[r.at], kb * T8_K, row);
          }
        }
      }
      if (!ok && (CG == 1 || !tokens || crank == 0)) {
        // let the copies already issued land before the CTA can exit (tokens: before the pair can)
        const uint32_t first = it > stages ? it - stages : 0;
        for (uint32_t j = first; j < it; ++j) {
          volatile uint32_t never = 0;
          mbar_wait_suspended(&got[j % stages], (j / stages) & 1u, &never, nullptr, 0);
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp goes through the loop, so that what an MMA takes stays in uniform registers; one lane issues.
    if (crank == 0) {
      const uint32_t idesc = idesc_f16_f32(T8_ROWS * CG, uint32_t(p.tokens));
      // descriptors by adding to a ready one (the address field counts 16 bytes)
      const uint64_t desc0 = sdesc_sw128(smem_u32(smem_t), 16u);
      const uint64_t stage_step = uint64_t(uint32_t(p.t_bytes) >> 4);
      const uint64_t kblock = uint64_t((uint32_t(p.tokens / CG) * 128u) >> 4);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem_base, 0);
      Turn w{0, 0}, acc{0, 0};
      bool ok = true;
      for (int u = u_first; u < p.units && ok; u += u_step, acc.step(1, accs)) {
        bool go = mbar_wait_suspended(&tail->tempty[acc.at], acc.parity ^ 1u, abort_flag, p.err, 0x1200u);
        if (!__all_sync(0xffffffffu, go)) break;
        tc_fence_after();
        const uint32_t d_tmem = tm + T8_ACC_COL + acc.at * T8_TWO_ACC;
        for (int kb = 0; kb < k_stages; ++kb) {
          go = mbar_wait_suspended(&tail->tgot[w.at], w.parity, abort_flag, p.err, 0x1301u) &&
               mbar_wait_suspended(&tail->wide[w.at], w.parity, abort_flag, p.err, 0x1300u);
          if (!__all_sync(0xffffffffu, go)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t bd = desc0 + w.at * stage_step;
          const uint32_t at = tm + w.at * 64u;
          const int steps = (p.K - kb * T8_K + 15) / 16;
          if (elect_one()) {
            if (steps >= T8_K / 16) {
#pragma unroll
              for (int k = 0; k < T8_K / 16; ++k)
                umma_f16_ts<CG>(d_tmem, at + uint32_t(k) * 8u, bd + (k >> 2) * kblock + uint64_t((k & 3) * 2), idesc,
                                (k != 0 || kb != 0) ? 1u : 0u);
            } else {
              for (int k = 0; k < steps; ++k)
                umma_f16_ts<CG>(d_tmem, at + uint32_t(k) * 8u, bd + uint64_t(k >> 2) * kblock + uint64_t((k & 3) * 2),
                                idesc, (kb | k) != 0 ? 1u : 0u);
            }
            if (CG == 2) {
              umma_commit_pair_mc(&tail->wfree[w.at], 0x3);
              if (kb == k_stages - 1) umma_commit_pair_mc(&tail->tfull[acc.at], 0x3);
            } else {
              umma_commit(&tail->wfree[w.at]);
              if (kb == k_stages - 1) umma_commit(&tail->tfull[acc.at]);
            }
          }
          __syncwarp();
          w.step(1, T8_WIDE);
        }
      }
      // every MMA issued above has completed once this arrives
      if (elect_one()) {
        if (CG == 2) umma_commit_pair_mc(&tail->drain, 0x1); else umma_commit(&tail->drain);
      }
      __syncwarp();
      volatile uint32_t never = 0;
      mbar_wait_suspended(&tail->drain, 0, &never, p.err, 0x1400u);
    }
  } else if (warp >= 4 && warp < 4 + T8_EPI) {
    // ------------------------------------------------------------ epilogue
    // lanes are channels, columns tokens: a token's 32 channels go out as one coalesced store.  A warp takes
    // half of the tokens.
    const uint32_t quarter = warp & 3u;
    const int half = int(warp - 4u) >> 2;
    const int first = half == 0 ? 0 : (p.tokens / 2 + 15) / 16 * 16;
    const int end = half == 0 ? (p.tokens / 2 + 15) / 16 * 16 : p.tokens;
    // a unit's scales are loaded while the one before is written out
    float sb = 0.f, next_sb = 0.f, next_sa[4] = {};
    auto load_scales = [&](const Walk& at) {
      const int n = (at.group * CG + int(crank)) * T8_ROWS + int(quarter * 32u + lane);
      const int tok0 = at.tile * p.tokens + first, toks = min(end - first, p.M - tok0);
      next_sb = n < p.N ? __ldg(p.b_scale + n) : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        next_sa[j] = 32 * j + int(lane) < toks ? __ldg(p.a_scale + tok0 + 32 * j + lane) : 0.f;
    };
    Walk next(p, u_first);
    if (next.u < p.units) load_scales(next);
    Turn acc{0, 0};
    for (Walk at = next; at.u < p.units; at = next, acc.step(1, accs)) {
      const int n = (at.group * CG + int(crank)) * T8_ROWS + int(quarter * 32u + lane);
      const int tok0 = at.tile * p.tokens + first, toks = min(end - first, p.M - tok0);  // <= 128, may be below 1
      float* sa = tail->a_scale[warp - 4u];
      __syncwarp();  // the last unit's have been read
#pragma unroll
      for (int j = 0; j < 4; ++j) sa[32 * j + lane] = next_sa[j];
      sb = next_sb;
      __syncwarp();
      next.step(p, u_step, step_groups, step_tiles);
      if (next.u < p.units) load_scales(next);
      const bool got = mbar_wait_suspended(&tail->tfull[acc.at], acc.parity, abort_flag, p.err, 0x1500u);
      if (!__all_sync(0xffffffffu, got)) break;
      tc_fence_after();
      const uint32_t t_acc = tmem_base + ((quarter * 32u) << 16) + T8_ACC_COL + acc.at * T8_TWO_ACC + uint32_t(first);
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CG == 2 && crank != 0) mbar_arrive_remote_tc(mapa_u32(&tail->tempty[acc.at], 0));
          else mbar_arrive(&tail->tempty[acc.at]);
        }
      };
      OUT* out = reinterpret_cast<OUT*>(p.C) + int64_t(tok0) * p.ldc + n;
      const bool whole = __all_sync(0xffffffffu, n < p.N);
      // 16 tokens' values: (sum a_scale) b_scale, each product rounded once
      auto values = [&](int c, float (&v)[16]) {
        uint32_t raw[16];
        tmem_ld_32x32b_x16(t_acc + c, raw);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 f = *reinterpret_cast<const float4*>(sa + c + i);
          v[i] = __fmul_rn(__fmul_rn(__uint_as_float(raw[i]), f.x), sb);
          v[i + 1] = __fmul_rn(__fmul_rn(__uint_as_float(raw[i + 1]), f.y), sb);
          v[i + 2] = __fmul_rn(__fmul_rn(__uint_as_float(raw[i + 2]), f.z), sb);
          v[i + 3] = __fmul_rn(__fmul_rn(__uint_as_float(raw[i + 3]), f.w), sb);
        }
      };
      if (sizeof(OUT) == 2 && accs == 1) {
        // the accumulator is waited for: it goes to registers, 32 tokens at a time in the output's type, and the
        // last of them are stored when it has been given back (64 at a time spill: 2000 x 256 x 100000 171 us, not 145)
        uint16_t* o = reinterpret_cast<uint16_t*>(out);
#pragma unroll 1
        for (int h = 0; h < 128; h += 32) {
          uint32_t packed[16];
#pragma unroll
          for (int c = 0; c < 32; c += 16) {
            if (h + c < toks) {
              float v[16];
              values(h + c, v);
#pragma unroll
              for (int i = 0; i < 16; i += 2) packed[(c + i) / 2] = pack_out<OUT>(v[i], v[i + 1]);
            }
          }
          if (h == 96) release();
          if (h + 32 <= toks && whole) {
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              o[0] = uint16_t(packed[c / 2] & 0xFFFFu);
              o[p.ldc] = uint16_t(packed[c / 2] >> 16);
              o += 2 * p.ldc;
            }
          } else {
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              if (h + c < toks && n < p.N) o[0] = uint16_t(packed[c / 2] & 0xFFFFu);
              if (h + c + 1 < toks && n < p.N) o[p.ldc] = uint16_t(packed[c / 2] >> 16);
              o += 2 * p.ldc;
            }
          }
        }
      } else {
        if (toks < 1) release();
#pragma unroll 1
        for (int c = 0; c < toks; c += 16) {
          float v[16];
          values(c, v);
          if (c + 16 >= toks) release();
          if (c + 16 <= toks && whole) {
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              store_pair(out, out + p.ldc, v[i], v[i + 1]);
              out += 2 * p.ldc;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (c + i < toks && n < p.N) store_out(out, v[i]);
              out += p.ldc;
            }
          }
        }
      }
    }
  } else if (warp >= 4 + T8_EPI) {
    // ------------------------------------------------------------ widening
    // A thread takes a channel's 128 bytes of a stage (128-byte rows, 16-byte chunks swizzled by row) to 64
    // columns of its lane in tensor memory, two consecutive k a column.
    const uint32_t quarter = warp & 3u, row = quarter * 32u + lane;
    const uint32_t t_lane = tmem_base + ((quarter * 32u) << 16);
    const uint32_t set = (warp - 4u - T8_EPI) >> 2;
    const uint32_t total = u_first < p.units ? uint32_t((p.units - 1 - u_first) / u_step + 1) * uint32_t(k_stages) : 0;
    Turn r{set, 0}, w{set, 0};
    for (uint32_t it = set; it < total; it += T8_SETS) {
      bool go = mbar_wait_suspended(&tail->wgot[r.at], r.parity, abort_flag, p.err, 0x1600u);
      if (!__all_sync(0xffffffffu, go)) break;
      const uint8_t* src = smem + size_t(r.at) * T8_W_BYTES + row * 128u;
      uint4 v[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] = *reinterpret_cast<const uint4*>(src + ((uint32_t(c) ^ (row & 7u)) * 16u));
      __syncwarp();
      if (lane == 0) mbar_arrive(&tail->wempty[r.at]);
      go = mbar_wait_suspended(&tail->wfree[w.at], w.parity ^ 1u, abort_flag, p.err, 0x1700u);
      if (!__all_sync(0xffffffffu, go)) break;
      tc_fence_after();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t d[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          widen4(v[h * 4 + c].x, d[c * 8], d[c * 8 + 1]);
          widen4(v[h * 4 + c].y, d[c * 8 + 2], d[c * 8 + 3]);
          widen4(v[h * 4 + c].z, d[c * 8 + 4], d[c * 8 + 5]);
          widen4(v[h * 4 + c].w, d[c * 8 + 6], d[c * 8 + 7]);
        }
        tmem_st_32x32b_x32(t_lane + w.at * 64u + uint32_t(h) * 32u, d);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2 && crank != 0) mbar_arrive_remote_tc(mapa_u32(&tail->wide[w.at], 0));
        else mbar_arrive(&tail->wide[w.at]);
      }
      w.step(T8_SETS, T8_WIDE);
      r.step(T8_SETS, w_stages);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();  // no commit or remote arrival of the peer can still target this CTA
  tc_fence_after();
  if (warp == 1) {
    if (CG == 2) tmem_dealloc_pair(tmem_base, TMEM_COLS); else tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// ------------------------------------------------------------------ few tokens ---
// Up to F8_TOKENS tokens: bound by reading the weights once.  The lanes of a group walk a weight row's 16-byte
// pieces with the tokens' integers in shared memory, four products an instruction into exact 32-bit sums.
// A group is as wide as a row has pieces (32 lanes at most) and takes some rows at a time, so that each
// piece of the tokens serves all of them and their loads are in flight together.  Rows may start anywhere: a
// piece then comes from the two aligned ones that it lies in, shifted; the second is in L1, as the next lane's.
// Rows at a time, blocks on an SM and pieces in flight by measurement (us, 2880 x 201088, rows / blocks / pieces):
//   one token             8/3/1 91 (6.4 TB/s), 4/3/2 112, 4/4/2 100, 4/2/4 101, 2/4/4 100; 8/2/2 129
//   one, rows anywhere    2/4/4 109, 4/4/2 122, 8/3/1 136, 4/3/2 149, 4/2/4 184
//   four                  4/3/2 115, 4/2/4 129, 4/4/2 160, 8/3/1 190
//   four, rows anywhere   4/2/4 164, 8/3/1 178, 4/4/2 194, 2/4/4 205, 4/3/2 240
// Other heads, the choice and the best of the five: one token 4096 x 151936 109 / 104 (4/2/4), 1024 x 50257 12.1, 256 x 50257
// 5.1, 2880 x 8192 12.0 / 8.6 (4/2/4), 1024 x 8192 5.7 / 4.7 (few rows a block leave fewer of the SMs' slots empty there);
// rows anywhere 115, 13.9, 6.0 / 5.7, 10.1, 5.3; four 2880 x 8192 13.8 / 13.5, 1024 x 8192 6.7, 256 x 50257 6.9; four, rows
// anywhere 4096 x 151936 166, 1024 x 50257 24, 2880 x 8192 14.8, 1024 x 8192 7.4 / 7.2.
constexpr int F8_THREADS = 256;
constexpr int F8_TOKENS = 4;
constexpr int F8_MAX_SMEM = 64 * 1024;

template <int MT, bool ANY>
struct Few {
  static constexpr int kRows = MT == 1 ? (ANY ? 2 : 8) : 4;
  static constexpr int kPerSm = MT == 1 ? (ANY ? 4 : 3) : (ANY ? 2 : 3);
  static constexpr int kUnroll = MT == 1 ? (ANY ? 4 : 1) : (ANY ? 4 : 2);
};

template <bool ANY>
__device__ __forceinline__ uint4 load_piece(const int8_t* p, int left) {
  // the piece's 16 bytes from p on, of which `left` >= 1 belong to the row (what follows meets zeros)
  if (!ANY) return __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t off = uint32_t(reinterpret_cast<uintptr_t>(p) & 15u);
  const uint4* a = reinterpret_cast<const uint4*>(p - off);
  const uint4 x = __ldg(a);
  uint4 y = make_uint4(0, 0, 0, 0);
  if (off != 0 && int(16u - off) < left) y = __ldg(a + 1);
  const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  uint32_t v[5];
#pragma unroll
  for (int j = 0; j < 5; ++j) {
    const uint32_t lo = (off & 4u) ? w[j + 1] : w[j];
    const uint32_t hi = (off & 4u) ? w[j + 3 > 7 ? 7 : j + 3] : w[j + 2 > 7 ? 7 : j + 2];
    v[j] = (off & 8u) ? hi : lo;
  }
  const uint32_t bits = (off & 3u) * 8u;
  return make_uint4(__funnelshift_r(v[0], v[1], bits), __funnelshift_r(v[1], v[2], bits),
                    __funnelshift_r(v[2], v[3], bits), __funnelshift_r(v[3], v[4], bits));
}

template <int MT, bool ANY, class OUT>
__global__ void __launch_bounds__(F8_THREADS)
    kd_gemm8_few_kernel(const int8_t* __restrict__ A, int64_t lda, const float* __restrict__ a_scale,
                        const int8_t* __restrict__ B, int64_t ldb, const float* __restrict__ b_scale,
                        OUT* __restrict__ C, int64_t ldc, int M, int64_t N, int K, int group) {
  extern __shared__ uint4 tok[];  // [MT][pieces]: zeros behind K and behind the last token
  const int pieces = (K + 15) / 16;
  for (int i = threadIdx.x; i < MT * pieces * 16; i += F8_THREADS) {
    const int m = i / (pieces * 16), k = i - m * pieces * 16;
    reinterpret_cast<int8_t*>(tok)[i] = m < M && k < K ? A[m * lda + k] : int8_t(0);
  }
  __syncthreads();
  constexpr int F8_ROWS = Few<MT, ANY>::kRows;
  const int lane = threadIdx.x & 31, at = lane & (group - 1);
  const int groups = F8_THREADS / group;
  const int64_t step = int64_t(gridDim.x) * groups * F8_ROWS;
  for (int64_t n0 = (int64_t(blockIdx.x) * groups + threadIdx.x / group) * F8_ROWS; ; n0 += step) {
    // a warp's groups leave together: their sums are exchanged below
    if (!__any_sync(0xffffffffu, n0 < N)) break;
    int acc[F8_ROWS][MT];
#pragma unroll
    for (int r = 0; r < F8_ROWS; ++r)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[r][m] = 0;
    const int64_t last = N - 1;
#pragma unroll (Few<MT, ANY>::kUnroll)
    for (int c = at; c < pieces; c += group) {
      uint4 w[F8_ROWS];
#pragma unroll
      for (int r = 0; r < F8_ROWS; ++r) {
        const int64_t n = n0 + r < N ? n0 + r : last;  // rows behind the last: its own again, not stored
        w[r] = load_piece<ANY>(B + n * ldb + c * 16, K - c * 16);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const uint4 t = tok[m * pieces + c];
#pragma unroll
        for (int r = 0; r < F8_ROWS; ++r) {
          int s = acc[r][m];
          s = __dp4a(int(w[r].x), int(t.x), s);
          s = __dp4a(int(w[r].y), int(t.y), s);
          s = __dp4a(int(w[r].z), int(t.z), s);
          acc[r][m] = __dp4a(int(w[r].w), int(t.w), s);
        }
      }
    }
    for (int o = group >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int r = 0; r < F8_ROWS; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[r][m] += __shfl_xor_sync(0xffffffffu, acc[r][m], o);
    if (at == 0) {
#pragma unroll
      for (int r = 0; r < F8_ROWS; ++r) {
        if (n0 + r >= N) break;
        const float sb = __ldg(b_scale + n0 + r);
#pragma unroll
        for (int m = 0; m < MT; ++m)
          if (m < M) store_out(C + m * ldc + n0 + r, __fmul_rn(__fmul_rn(float(acc[r][m]), __ldg(a_scale + m)), sb));
      }
    }
  }
}

// ------------------------------------------------------------------ operands ---
// The tokens as fp16, rows of Kp (K to the next 64, zeros behind): small beside the weights, read by every
// tile.  A thread takes 8 elements; rows that start unaligned are read byte by byte.
__global__ void __launch_bounds__(256)
    kd_int8_tokens_kernel(const int8_t* __restrict__ A, int64_t lda, int M, int K, int Kp, int aligned8,
                          uint4* __restrict__ out) {
  const int per_row = Kp / 8;
  const int64_t total = int64_t(M) * per_row;
  for (int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; i < total; i += int64_t(gridDim.x) * blockDim.x) {
    const int64_t m = i / per_row;
    const int k = int(i - m * per_row) * 8;
    const int8_t* src = A + m * lda + k;
    uint32_t w[2] = {0, 0};
    if (aligned8 && k + 8 <= K) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
      w[0] = v.x;
      w[1] = v.y;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (k + j < K) w[j >> 2] |= uint32_t(uint8_t(src[j])) << (8 * (j & 3));
    }
    uint4 o;
    widen4(w[0], o.x, o.y);
    widen4(w[1], o.z, o.w);
    out[i] = o;
  }
}

// Weights whose rows do not start on 16-byte boundaries, copied to rows that do (K to the next 16).  A thread
// makes 16 bytes from the two 4-byte-aligned words either side of each of its four.
__global__ void __launch_bounds__(256)
    kd_int8_rows_kernel(const int8_t* __restrict__ B, int64_t ldb, int64_t N, int K, int Kp, uint4* __restrict__ out) {
  const int per_row = Kp / 16;
  const int64_t total = N * per_row;
  for (int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; i < total; i += int64_t(gridDim.x) * blockDim.x) {
    const int64_t n = i / per_row;
    const int k = int(i - n * per_row) * 16;
    const int8_t* src = B + n * ldb + k;
    const int left = K - k;  // elements of this row from k on
    uint32_t o[4];
    if (left >= 20) {
      // the word behind the sixteenth element still lies in this row
      const uint32_t off = uint32_t(reinterpret_cast<uintptr_t>(src) & 3u);
      const uint32_t* w = reinterpret_cast<const uint32_t*>(src - off);
      uint32_t v[5];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __ldg(w + j);
      v[4] = off ? __ldg(w + 4) : 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = __funnelshift_r(v[j], v[j + 1], off * 8u);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o[j] = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (j * 4 + b < left) o[j] |= uint32_t(uint8_t(src[j * 4 + b])) << (8 * b);
      }
    }
    out[i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// ------------------------------------------------------------------ quantisation ---
// A row is shared by W warps of a block, each thread holding 64 bytes of it (vectors of VE elements) in registers
// between the two sweeps (128: 8192 x 4096 bf16 32 us against 27); what a longer row has beyond that is read twice.  Bound by HBM: an element read and a byte
// written.  A row that holds a NaN or an infinity has scale NaN and integers 0, a row of zeros scale 0.
//
// x times the rounded 1 / s is within 2^-23 of the quotient, 127 at most: its nearest whole number is the
// quotient's unless it lies within 1.6e-5 of a half.  Then x / s is rounded correctly to fp32, and where that lands
// on a tie, the sign of what the division left over says on which side the quotient lies.
constexpr float kSureOff = 0.49998f;
constexpr float kRoundMagic = 12582912.f;  // 1.5 * 2^23: whole numbers in the low bits of the sum

__device__ __noinline__ int quantized_near_half(float x, float s) {
  const float v = __fdiv_rn(x, s);
  float r = rintf(v);
  if (fabsf(v - truncf(v)) == 0.5f) {
    const float up = s < 1.f ? 16777216.f : 1.f;       // so that nothing below is rounded away
    const float rest = fmaf(-v, s * up, x * up);       // exact: x - v s
    if (rest != 0.f) r = rest > 0.f ? ceilf(v) : floorf(v);
  }
  return int(fminf(fmaxf(r, -127.f), 127.f));
}

// N elements' integers, four to a word.  inv 0: every element by division (a scale whose reciprocal fp32 does not
// hold).  One test for all of them first, as few lie near a half.
template <int N, class X>
__device__ __forceinline__ void quantize_vec(const X& x, float s, float inv, uint32_t* out) {
  float m[N], far = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float v = x.get(i);
    m[i] = fmaf(v, inv, kRoundMagic);
    far = fmaxf(far, fabsf(fmaf(v, inv, kRoundMagic - m[i])));
  }
  if (!(far < kSureOff) || inv == 0.f) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!(fabsf(fmaf(x.get(i), inv, kRoundMagic - m[i])) < kSureOff) || inv == 0.f)
        m[i] = __int_as_float(quantized_near_half(x.get(i), s));
  }
  uint32_t q[(N + 3) / 4 * 4];
#pragma unroll
  for (int i = 0; i < (N + 3) / 4 * 4; ++i) q[i] = i < N ? __float_as_uint(m[i < N ? i : 0]) : 0u;
#pragma unroll
  for (int i = 0; i < (N + 3) / 4; ++i)
    out[i] = __byte_perm(__byte_perm(q[4 * i], q[4 * i + 1], 0x0040), __byte_perm(q[4 * i + 2], q[4 * i + 3], 0x0040), 0x5410);
}

template <class T, int VE>
struct QVec {
  uint32_t w[VE * sizeof(T) < 4 ? 1 : VE * sizeof(T) / 4];
  __device__ __forceinline__ void load(const T* p) {
    if (VE * sizeof(T) == 16) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if (VE * sizeof(T) == 8) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = v.x; w[1] = v.y;
    } else if (sizeof(T) == 2) {
      w[0] = __ldg(reinterpret_cast<const uint16_t*>(p));
    } else {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (uint32_t& x : w) x = 0;
  }
  __device__ __forceinline__ float get(int i) const;
  // the largest magnitude so far, as bits (of one element, or of two 16-bit ones side by side): infinities and
  // NaNs lie above every number
  __device__ __forceinline__ uint32_t largest(uint32_t most) const {
#pragma unroll
    for (uint32_t x : w) most = sizeof(T) == 4 ? max(most, x & 0x7FFFFFFFu) : __vmaxu2(most, x & 0x7FFF7FFFu);
    return most;
  }
  // those bits as fp32's
  __device__ __forceinline__ static uint32_t as_f32(uint32_t most) {
    if (sizeof(T) == 4) return most;
    const uint32_t h = max(most & 0xFFFFu, most >> 16);
    return std::is_same<T, __half>::value ? __float_as_uint(__half2float(__ushort_as_half(uint16_t(h)))) : h << 16;
  }
};
template <class T, int VE>
__device__ __forceinline__ float QVec<T, VE>::get(int i) const {
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(w[i]);
  } else {
    const uint32_t h = (i & 1) ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu;
    if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half(uint16_t(h)));
    else return __uint_as_float(h << 16);
  }
}

constexpr int Q_THREADS = 256;
template <class T>
constexpr int kQEach = 64 / sizeof(T);  // elements that a thread holds

template <class T, int VE, int W>
__global__ void __launch_bounds__(Q_THREADS)
    kd_quantize_kernel(const T* __restrict__ x, int64_t N, int64_t d, int64_t ld, int8_t* __restrict__ q, int64_t ldq,
                       float* __restrict__ scale) {
  constexpr int NV = kQEach<T> / VE, ROWS = Q_THREADS / 32 / W, LANES = 32 * W;
  __shared__ uint32_t part[2][Q_THREADS / 32];
  const int warp = threadIdx.x >> 5, group = warp / W;
  const int lane = threadIdx.x - group * LANES;
  const int nv = int(d / VE);  // VE > 1 only where it divides d
  int turn = 0;
  // a row's warps go through the loop together, and wait for nobody else
  for (int64_t n = int64_t(blockIdx.x) * ROWS + group; n < N; n += int64_t(gridDim.x) * ROWS, turn ^= 1) {
    const T* row = x + n * ld;
    QVec<T, VE> v[NV];
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int at = lane + j * LANES;
      if (at < nv) v[j].load(row + at * VE); else v[j].zero();
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) most = v[j].largest(most);
    for (int at = lane + NV * LANES; at < nv; at += LANES) {
      QVec<T, VE> a;
      a.load(row + at * VE);
      most = a.largest(most);
    }
    most = __reduce_max_sync(0xffffffffu, QVec<T, VE>::as_f32(most));
    if (W > 1) {
      if ((threadIdx.x & 31) == 0) part[turn][warp] = most;
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(LANES) : "memory");
#pragma unroll
      for (int w = 0; w < W; ++w) most = max(most, part[turn][group * W + w]);
    }
    const float s = most < 0x7F800000u ? __fdiv_rn(__uint_as_float(most), 127.f) : __int_as_float(0x7FC00000);
    const float inv = s > 1e-37f ? 1.f / s : 0.f;
    const bool none = !(s > 0.f);
    if (lane == 0) scale[n] = s;
    int8_t* out = q + n * ldq;
    auto put = [&](const QVec<T, VE>& a, int at) {
      uint32_t o[(VE + 3) / 4] = {};
      if (!none) quantize_vec<VE>(a, s, inv, o);
      if constexpr (VE == 8) *reinterpret_cast<uint2*>(out + at * VE) = make_uint2(o[0], o[1]);
      else if constexpr (VE == 4) *reinterpret_cast<uint32_t*>(out + at * VE) = o[0];
      else if constexpr (VE == 2) *reinterpret_cast<uint16_t*>(out + at * VE) = uint16_t(o[0]);
      else out[at] = int8_t(o[0]);
    };
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int at = lane + j * LANES;
      if (at < nv) put(v[j], at);
    }
    for (int at = lane + NV * LANES; at < nv; at += LANES) {
      QVec<T, VE> a;
      a.load(row + at * VE);
      put(a, at);
    }
  }
}

template <class T, int VE, int W>
cudaError_t launch_quantize_rows(const T* x, int64_t N, int64_t d, int64_t ld, int8_t* q, int64_t ldq, float* scale,
                                 cudaStream_t s) {
  constexpr int ROWS = Q_THREADS / 32 / W;
  const int64_t blocks = (N + ROWS - 1) / ROWS, most = int64_t(16) * gemm_max_grid();
  kd_quantize_kernel<T, VE, W><<<unsigned(blocks < most ? blocks : most), Q_THREADS, 0, s>>>(x, N, d, ld, q, ldq, scale);
  return cudaGetLastError();
}

// Warps to a row: as few as hold it in registers, so that short rows do not leave threads without work.
template <class T, int VE>
cudaError_t launch_quantize_width(const T* x, int64_t N, int64_t d, int64_t ld, int8_t* q, int64_t ldq, float* scale,
                                  cudaStream_t s) {
  if (d <= 32 * kQEach<T>) return launch_quantize_rows<T, VE, 1>(x, N, d, ld, q, ldq, scale, s);
  if (d <= 64 * kQEach<T>) return launch_quantize_rows<T, VE, 2>(x, N, d, ld, q, ldq, scale, s);
  if (d <= 128 * kQEach<T>) return launch_quantize_rows<T, VE, 4>(x, N, d, ld, q, ldq, scale, s);
  return launch_quantize_rows<T, VE, 8>(x, N, d, ld, q, ldq, scale, s);
}

template <class T>
cudaError_t launch_quantize_typed(const void* x, int64_t N, int64_t d, int64_t ld, int8_t* q, int64_t ldq,
                                  float* scale, cudaStream_t s) {
  // vectors of 16 or 8 bytes where every row allows them
  constexpr int V16 = 16 / sizeof(T), V8 = 8 / sizeof(T);
  const T* p = static_cast<const T*>(x);
  auto fits = [&](int ve) {
    return aligned(x, ve * sizeof(T)) && aligned(q, size_t(ve)) && d % ve == 0 &&
           (N == 1 || (ld % ve == 0 && ldq % ve == 0));
  };
  if (fits(V16)) return launch_quantize_width<T, V16>(p, N, d, ld, q, ldq, scale, s);
  if (fits(V8)) return launch_quantize_width<T, V8>(p, N, d, ld, q, ldq, scale, s);
  return launch_quantize_width<T, 1>(p, N, d, ld, q, ldq, scale, s);
}

// ------------------------------------------------------------------ host side ---

template <int CG, class OUT>
cudaError_t launch_t8(const T8Problem& p, const CUtensorMap& tw, const CUtensorMap& tt, cudaStream_t s) {
  static PerDevice<int> resident;  // clusters (CTAs) on the device at once
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(T8_THREADS, 1, 1);
  cfg.dynamicSmemBytes = T8_SMEM;
  cfg.stream = s;
  int most = 1;
  const int rc = resident.get(dev, &most, [&](int, int* v) {
    const cudaError_t r =
        cudaFuncSetAttribute(kd_gemm8_kernel<CG, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, T8_SMEM);
    if (r != cudaSuccess) return int(r);
    *v = gemm_max_grid() / CG;
    if (CG == 2) {
      cudaLaunchConfig_t q = cfg;
      q.gridDim = dim3(unsigned(gemm_max_grid() / 2 * 2), 1, 1);
      q.stream = nullptr;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, kd_gemm8_kernel<CG, OUT>, &q) == cudaSuccess && n >= 1) *v = n;
    }
    return 0;
  });
  if (rc != 0) return rc > 0 ? cudaError_t(rc) : cudaErrorInvalidDevice;
  cfg.gridDim = dim3(unsigned((p.units < most ? p.units : most) * CG), 1, 1);
  e = cudaLaunchKernelEx(&cfg, kd_gemm8_kernel<CG, OUT>, tw, tt, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int CG>
cudaError_t launch_t8_typed(int dtype, const T8Problem& p, const CUtensorMap& tw, const CUtensorMap& tt,
                            cudaStream_t s) {
  prof_before("kd_gemm8", s);
  const cudaError_t e = dtype == KD_F32   ? launch_t8<CG, float>(p, tw, tt, s)
                        : dtype == KD_F16 ? launch_t8<CG, __half>(p, tw, tt, s)
                                          : launch_t8<CG, uint16_t>(p, tw, tt, s);
  prof_after(s);
  return e;
}

// Tokens up to which single CTAs compute a tile; a pair halves the loads of more.
constexpr int T8_SINGLE = 64;

// Whether the tokens are few, and fit into a block's shared memory.  One always; up to F8_TOKENS where the tensor
// cores' way would copy the weights to aligned rows first (four tokens, 2880 x 201088: 164 us against 287), or
// where the weights are few, so that its longer start counts (two tokens, four, that way; us, weights not in the L2:
// 256 x 50257 6.2, 7.2, 9.4; 1024 x 8192 5.4, 6.4, 8.9; 2880 x 4096 11.3, 12.2, 14.0; 4096 x 5000 13.3, 15.6, 17.1; 2880 x 8192,
// 24 million, 12.2, 13.8, 14.4; 2880 x 16000 20.0, 20.3, 15.7; 4096 x 32000 35.6, 38.1, 31.6; 2880 x 201088 118, 117, 102.
// K = 1024 turns later: 1024 x 50257 14.2, 15.1, 16.5).
constexpr int64_t F8_WEIGHTS = 24000000;

bool int8_few(int64_t M, int64_t N, int64_t K, bool aligned_rows) {
  if (M > F8_TOKENS || (M > 1 && aligned_rows && N * K > F8_WEIGHTS)) return false;
  return (M <= 1 ? 1 : M <= 2 ? 2 : 4) * ((K + 15) / 16 * 16) <= F8_MAX_SMEM;
}

struct I8Layout {
  size_t tokens, weights, total;
  int64_t Kp, Kw;
};

I8Layout int8_layout(int64_t M, int64_t N, int64_t K, bool aligned_rows) {
  I8Layout L{};
  L.total = sizeof(Ctrl);
  if (int8_few(M, N, K, aligned_rows)) return L;
  L.Kp = (K + 63) / 64 * 64;
  L.Kw = (K + 15) / 16 * 16;
  L.tokens = sizeof(Ctrl);
  L.weights = align_up(L.tokens + size_t(M) * size_t(L.Kp) * 2, 256);
  L.total = aligned_rows ? L.weights : align_up(L.weights + size_t(N) * size_t(L.Kw), 256);
  return L;
}

template <int MT, bool ANY, class OUT>
cudaError_t launch_few(const int8_t* A, int64_t lda, const float* a_scale, const int8_t* B, int64_t ldb,
                       const float* b_scale, void* C, int64_t ldc, int64_t M, int64_t N, int64_t K, cudaStream_t s) {
  static PerDevice<int> attr_done;
  const cudaError_t e = smem_attr_once(attr_done, reinterpret_cast<const void*>(kd_gemm8_few_kernel<MT, ANY, OUT>),
                                       F8_MAX_SMEM);
  if (e != cudaSuccess) return e;
  const int64_t pieces = (K + 15) / 16;
  int group = 32;
  while (group > 1 && group / 2 >= pieces) group /= 2;
  const int64_t per_block = int64_t(F8_THREADS / group) * Few<MT, ANY>::kRows;
  const int64_t blocks = (N + per_block - 1) / per_block, most = int64_t(Few<MT, ANY>::kPerSm) * gemm_max_grid();
  kd_gemm8_few_kernel<MT, ANY, OUT><<<unsigned(blocks < most ? blocks : most), F8_THREADS, size_t(MT) * pieces * 16, s>>>(
      A, lda, a_scale, B, ldb, b_scale, static_cast<OUT*>(C), ldc, int(M), N, int(K), group);
  return cudaGetLastError();
}

template <int MT, bool ANY>
cudaError_t launch_few_typed(const int8_t* A, int64_t lda, const float* a_scale, const int8_t* B, int64_t ldb,
                             const float* b_scale, void* C, int dtype, int64_t ldc, int64_t M, int64_t N, int64_t K,
                             cudaStream_t s) {
  if (dtype == KD_F32) return launch_few<MT, ANY, float>(A, lda, a_scale, B, ldb, b_scale, C, ldc, M, N, K, s);
  if (dtype == KD_F16) return launch_few<MT, ANY, __half>(A, lda, a_scale, B, ldb, b_scale, C, ldc, M, N, K, s);
  return launch_few<MT, ANY, uint16_t>(A, lda, a_scale, B, ldb, b_scale, C, ldc, M, N, K, s);
}

template <int MT>
cudaError_t launch_few_any(bool rows16, const int8_t* A, int64_t lda, const float* a_scale, const int8_t* B,
                           int64_t ldb, const float* b_scale, void* C, int dtype, int64_t ldc, int64_t M, int64_t N,
                           int64_t K, cudaStream_t s) {
  return rows16 ? launch_few_typed<MT, false>(A, lda, a_scale, B, ldb, b_scale, C, dtype, ldc, M, N, K, s)
                : launch_few_typed<MT, true>(A, lda, a_scale, B, ldb, b_scale, C, dtype, ldc, M, N, K, s);
}

unsigned blocks_for(int64_t work, int per_sm) {
  const int64_t b = (work + 255) / 256, most = int64_t(per_sm) * gemm_max_grid();
  return unsigned(b < 1 ? 1 : b < most ? b : most);
}

}  // namespace

cudaError_t launch_gemm_int8(const int8_t* A, int64_t lda, const float* a_scale, const int8_t* B, int64_t ldb,
                             const float* b_scale, void* C, int dtype, int64_t ldc, int64_t M, int64_t N, int64_t K,
                             uint8_t* ws, uint32_t* err, cudaStream_t s) {
  const bool rows16 = aligned(B, 16) && ldb % 16 == 0;
  if (int8_few(M, N, K, rows16)) {
    prof_before("kd_gemm8_few", s);
    const cudaError_t f =
        M <= 1   ? launch_few_any<1>(rows16, A, lda, a_scale, B, ldb, b_scale, C, dtype, ldc, M, N, K, s)
        : M <= 2 ? launch_few_any<2>(rows16, A, lda, a_scale, B, ldb, b_scale, C, dtype, ldc, M, N, K, s)
                 : launch_few_any<4>(rows16, A, lda, a_scale, B, ldb, b_scale, C, dtype, ldc, M, N, K, s);
    prof_after(s);
    return f;
  }
  const I8Layout L = int8_layout(M, N, K, rows16);
  uint4* tokens = reinterpret_cast<uint4*>(ws + L.tokens);
  prof_before("kd_int8_tokens", s);
  kd_int8_tokens_kernel<<<blocks_for(M * L.Kp / 8, 8), 256, 0, s>>>(A, lda, int(M), int(K), int(L.Kp),
                                                                  aligned(A, 8) && lda % 8 == 0, tokens);
  prof_after(s);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const void* weights = B;
  uint64_t w_stride = uint64_t(ldb);
  if (!rows16) {
    if ((e = launch_int8_rows(B, ldb, N, K, L.Kw, ws + L.weights, s)) != cudaSuccess) return e;
    weights = ws + L.weights;
    w_stride = uint64_t(L.Kw);
  }

  T8Problem p{};
  p.M = int(M); p.N = int(N); p.K = int(K);
  // Short reductions leave the draining of a large accumulator waited for too often.  us with at most 256 / 128
  // tokens a tile: 2000 x 100000, K = 256 158 / 146, K = 512 205 / 176, K = 768 250 / 240; 2000 x 50000, K = 1024
  // 154 / 159, K = 1536 201 / 224.
  const int most = K <= T8_SHORT_K ? T8_TWO_ACC : T8_MAX_TOKENS;
  p.token_tiles = int((M + most - 1) / most);
  const int64_t even = (M + p.token_tiles - 1) / p.token_tiles;  // tiles of nearly the same size
  const int cg = even <= T8_SINGLE ? 1 : 2;
  p.tokens = int((even + 16 * cg - 1) / (16 * cg) * (16 * cg));
  p.t_bytes = p.tokens / cg * 256;
  p.w_stages = (T8_SMEM - 1024 - int(sizeof(T8Tail)) - T8_WIDE * p.t_bytes) / T8_W_BYTES / T8_SETS * T8_SETS;
  if (p.w_stages > T8_MAX_STAGES) p.w_stages = T8_MAX_STAGES;
  const int64_t channel_tiles = (N + T8_ROWS - 1) / T8_ROWS;
  p.units = int((channel_tiles + cg - 1) / cg * p.token_tiles);
  p.a_scale = a_scale; p.b_scale = b_scale;
  p.C = C; p.ldc = ldc;
  p.err = err;
  alignas(64) CUtensorMap tw, tt;
  if (!make_tmap_2d_u8(&tw, weights, uint64_t(K), uint64_t(N), w_stride, T8_K, T8_ROWS) ||
      !make_tmap_mn2_bf16(&tt, tokens, uint64_t(L.Kp), uint64_t(M), uint64_t(L.Kp) * 2, uint32_t(p.tokens / cg)))
    return cudaErrorInvalidValue;
  return cg == 1 ? launch_t8_typed<1>(dtype, p, tw, tt, s) : launch_t8_typed<2>(dtype, p, tw, tt, s);
}

cudaError_t launch_int8_rows(const int8_t* B, int64_t ldb, int64_t N, int64_t K, int64_t Kw, void* out,
                             cudaStream_t s) {
  prof_before("kd_int8_rows", s);
  kd_int8_rows_kernel<<<blocks_for(N * (Kw / 16), 16), 256, 0, s>>>(B, ldb, N, int(K), int(Kw), static_cast<uint4*>(out));
  prof_after(s);
  return cudaGetLastError();
}

bool gemm_int8_copies_rows(int64_t M, int64_t N, int64_t K) { return !int8_few(M, N, K, false); }

size_t gemm_int8_scratch(int64_t M, int64_t N, int64_t K, bool aligned_rows) {
  return int8_layout(M, N, K, aligned_rows).total;
}

cudaError_t launch_quantize_int8(const void* x, int dtype, int64_t N, int64_t d, int64_t ld, int8_t* q, int64_t ldq,
                                 float* scale, cudaStream_t s) {
  prof_before("kd_quantize_int8", s);
  const cudaError_t e = dtype == KD_F32   ? launch_quantize_typed<float>(x, N, d, ld, q, ldq, scale, s)
                        : dtype == KD_F16 ? launch_quantize_typed<__half>(x, N, d, ld, q, ldq, scale, s)
                                          : launch_quantize_typed<uint16_t>(x, N, d, ld, q, ldq, scale, s);
  prof_after(s);
  return e;
}

}  // namespace kd
