// What a thread of the chunk attention does with its (token, head) row: the weights of a
// block of 64 positions from its scores, and the row's result.  Shared by the kernels that
// differ in how they bring scores and value products about.
#pragma once
#include <cuda_bf16.h>

#include "smla_chunk.h"
#include "smla_ptx.cuh"

namespace smla {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994530942f;
// The running maximum is raised only when a score passes it by 2^8: sums stay well inside
// 32 bits, a weight's bf16 rounding is relative, and most blocks rescale nothing.
constexpr float kHeadroom = 8.f;
constexpr long long kWaitLimit = 2000000000ll;     // SM clocks, ~1 s

// A wait that gives up on its limit or when another role has.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* stop, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*stop) return false;
    if (clock64() - t0 > kWaitLimit) {
      *stop = 1;
      atomicCAS(status, 0, SMLA_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}
// The same for a whole warp: one verdict for its lanes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* stop, int* status) {
  return __all_sync(0xffffffffu, wait(bar, parity, stop, status));
}

// What may be done to a score x = q . k besides the scale: a cap and a distance bias (both
// in units of log2).
//
// cap tanh(z), z = scale x / cap: up to |z| = 1/4 by tanh's series up to z^9 (the next term is
// 9e-9 of the first), past it 1 - 2 / (1 + e^(2 z)), whose difference would lose small values'
// digits (a lse of a few positions was off by 5e-6).  Usual scores are far below the cap, and then
// only the series is worked out, two scores an instruction (the mixed batch of 16 heads: 59.3 us; 71.8
// with one, 58.5 by the exponential form).  It is one in z itself: with the powers of scale / cap in
// its coefficients, a product less, they overflow for a cap far below the scale (0 times infinity
// where the score is 0) and vanish for one far above.  The product costs half a microsecond of that batch.
struct ScoreMods {
  float scale2, cap2, z1, inner, most;     // scale, cap, scale / cap, 2 z1, and the x of z = 1/4; cap2 0: none
  __device__ __forceinline__ explicit ScoreMods(const ChunkArgs& a)
      : scale2(a.scale * kLog2e), cap2(0.f), z1(0.f), inner(0.f), most(0.f) {
    if (a.cap > 0.f) {
      constexpr float kMost = 3.402823466e38f;      // what passes it stays finite: 0 times it is 0
      cap2 = fminf(a.cap * kLog2e, 0.5f * kMost);
      z1 = fminf(a.scale / a.cap, kMost);
      inner = fminf(2.f * kLog2e * z1, kMost);
      most = 0.25f / z1;
    }
  }
  __device__ __forceinline__ void series(float* x, float* y) const {
    const Two v(*x, *y), z = v * Two(z1), u = z * z, s = v * Two(scale2);
    const Two p = fma2(fma2(fma2(u, Two(62.f / 2835.f), Two(-17.f / 315.f)), u, Two(2.f / 15.f)), u, Two(-1.f / 3.f));
    fma2(s * u, p, s).get(x, y);
  }
  // The scores v of a thread; away(c): slope and distance of score c.
  template <int N, class Away>
  __device__ __forceinline__ void operator()(float (&v)[N], Away away) const {
    if (cap2 > 0.f) {
      float top = 0.f;
#pragma unroll
      for (int c = 0; c < N; ++c) top = fmaxf(top, fabsf(v[c]));
      if (!__any_sync(0xffffffffu, top > most)) {
#pragma unroll
        for (int c = 0; c < N; c += 2) series(&v[c], &v[c + 1]);
      } else {
#pragma unroll
        for (int c = 0; c < N; c += 2) {
          float near[2] = {v[c], v[c + 1]};
          series(&near[0], &near[1]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float far = cap2 - __fdividef(2.f * cap2, 1.f + exp2_fast(v[c + i] * inner));
            v[c + i] = fabsf(v[c + i]) > most ? far : near[i];
          }
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < N; ++c) v[c] *= scale2;
    }
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const float2 d = away(c);
      v[c] = fmaf(-d.x, fabsf(d.y), v[c]);
    }
  }
};

// The positions of the 64 from s0 on, of those in `mapped`, that lie in [lo, hi).
__device__ __forceinline__ unsigned long long seen_of(unsigned long long mapped, int s0, int lo, int hi) {
  const int c0 = max(0, lo - s0), c1 = min(64, hi - s0);
  if (c0 <= 0 && c1 >= 64) return mapped;
  return c1 > c0 ? mapped & (~0ull << c0) & (~0ull >> (64 - c1)) : 0ull;
}

// MODS: scores may be capped or biased by distance.
template <bool MODS>
struct RowState {
  // l sums the weights for the lse, lr their bf16 roundings, which the value product uses:
  // normalised by lr, a rounding moves out by its weight times v - out only
  float m = -INFINITY, l = 0.f, lr = 0.f;
  int lo = 0, hi = 0, pos = 0;       // visible positions, own position
  ScoreMods mods;
  float slope2 = 0.f;

  __device__ __forceinline__ RowState(const ChunkArgs& a, const ChunkPlan& plan, const int4& tile, int row,
                                      bool mine)
      : mods(a) {
    if (!mine) return;
    const int tok = (tile.y + row) / a.H;
    visible(a, tile.x, tok, plan.seq_len[tile.x], &lo, &hi, &pos);
    if (MODS && a.slopes != nullptr) slope2 = a.slopes[tile.y + row - tok * a.H] * kLog2e;
  }

  // The row's scores v of the block that starts at position s0 -> its weights p (bf16
  // pairs).  rows: the block's mapped positions, and those whose row is not finite.
  // Returns the factor by which earlier results of the row shrink.
  __device__ __forceinline__ float weights(float (&v)[64], int s0, const ulonglong2& rows, uint32_t (&p)[32]) {
    const float scale2 = mods.scale2;
    if constexpr (MODS) {
      const float from = static_cast<float>(pos - s0);
      mods(v, [&](int c) { return make_float2(slope2, from - static_cast<float>(c)); });
    }
    const unsigned long long seen = seen_of(rows.x, s0, lo, hi);
    if (__any_sync(0xffffffffu, seen != ~0ull)) {
#pragma unroll
      for (int c = 0; c < 64; ++c)
        if (!((seen >> c) & 1)) v[c] = -INFINITY;
    }
    float top = fmaxf(v[0], v[1]);
#pragma unroll
    for (int c = 2; c < 64; ++c) top = fmaxf(top, v[c]);
    if constexpr (!MODS) top *= scale2;
    float alpha = 1.f;
    if (top > m + kHeadroom || (m == -INFINITY && top > m)) {
      alpha = exp2_fast(m - top);     // 0 while m is -inf
      m = top;
      l *= alpha;
      lr *= alpha;
    }
    const float shift = m == -INFINITY ? 0.f : m;
    float sum0 = 0.f, sum1 = 0.f, rsum0 = 0.f, rsum1 = 0.f;
#pragma unroll
    for (int c = 0; c < 64; c += 2) {
      const float e0 = exp2_fast(MODS ? v[c] - shift : fmaf(v[c], scale2, -shift));
      const float e1 = exp2_fast(MODS ? v[c + 1] - shift : fmaf(v[c + 1], scale2, -shift));
      sum0 += e0;
      sum1 += e1;
      p[c / 2] = pack_bf16(e0, e1);
      rsum0 += __uint_as_float(p[c / 2] << 16);
      rsum1 += __uint_as_float(p[c / 2] & 0xffff0000u);
    }
    l += sum0 + sum1;
    lr += rsum0 + rsum1;
    // a row with NaN or infinities is held as zeros, since it would reach every row of the
    // tile through the value product; the rows that see it become NaN here
    if (seen & rows.y) l = lr = __uint_as_float(0x7fffffffu);
    return alpha;
  }
};

// Row r's weights into the 128-byte rows of P (K-major, 128-byte swizzle).
__device__ __forceinline__ void store_weights(uint32_t p_base, int r, const uint32_t (&p)[32]) {
#pragma unroll
  for (int u = 0; u < 8; ++u)
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(p_base + r * 128 + ((u ^ (r & 7)) << 4)),
                 "r"(p[4 * u]), "r"(p[4 * u + 1]), "r"(p[4 * u + 2]), "r"(p[4 * u + 3])
                 : "memory");
}

// `count` columns of the warp's rows of O times alpha, unless it is 1 for all of them.
// O is rescaled only where a row's maximum rises by more than kHeadroom, so seldom.
__device__ __forceinline__ void rescale_rows(uint32_t tO, float alpha, int first = 0, int count = kNope) {
  if (!__any_sync(0xffffffffu, alpha != 1.f)) return;
#pragma unroll 1
  for (int c = first; c < first + count; c += 32) {
    float o[32];
    tmem_ld32(tO + c, o);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 32; ++k) o[k] *= alpha;
    tmem_st16(tO + c, o);
    tmem_st16(tO + c + 16, o + 16);
  }
  tmem_wait_st();
}

// 1 / sum and lse of a row with maximum m, sum l and sum of rounded weights lr; a row that
// saw nothing gives 0 and -inf, NaN stays NaN.
__device__ __forceinline__ float inverse_sum(float l, float lr) { return l == 0.f ? 0.f : 1.f / lr; }
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2; }

// The results of a warp's rows row0 .. + 31 of the tile (lane = row): final (`whole`), or
// partial into `slot`.  inv: 1 / sum of the lane's row.  They pass through 4 KB of shared
// memory (`stage`), so that consecutive lanes write 128 consecutive bytes of a row: written
// by the lane that holds it, 16 bytes of 32 rows at a time, a tile took 14 us.
template <int TILE_ROWS>
__device__ __forceinline__ void store_rows(const ChunkArgs& a, const ChunkPlan& plan, float inv, float lse,
                                           uint32_t tO, const int4& tile, int row0, bool whole, int slot,
                                           uint32_t stage) {
  const int lane = threadIdx.x & 31;
  const int64_t orow = static_cast<int64_t>(tile.y) + row0;
  const int64_t prow = static_cast<int64_t>(slot) * TILE_ROWS + row0;
  const int live = min(32, tile.z - row0);         // rows of the warp that the tile has
  // 16-byte unit u of row r, so that 8 rows' same units and a row's units lie in different banks
  auto place = [&](int r, int u) { return stage + r * 128 + ((u ^ (r & 7)) << 4); };
  auto put = [&](int u, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(place(lane, u)), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
  };
  // the staged bytes of each row to base + row * pitch
  auto flush = [&](char* base, int64_t pitch) {
    __syncwarp();
    const int unit = lane & 7;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 4 + lane / 8;
      uint4 v;
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                   : "r"(place(r, unit))
                   : "memory");
      if (r < live) *reinterpret_cast<uint4*>(base + r * pitch + 16 * unit) = v;
    }
    __syncwarp();
  };
#pragma unroll 1
  for (int c = 0; c < kNope; c += 32) {
    float o[32];
    tmem_ld32(tO + c, o);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 32; ++k) o[k] *= inv;
    if (whole) {
      // 64 bytes a row: half of a staged row
      const int u0 = (c / 32 % 2) * 4;
#pragma unroll
      for (int k = 0; k < 32; k += 8)
        put(u0 + k / 8, pack_bf16(o[k], o[k + 1]), pack_bf16(o[k + 2], o[k + 3]), pack_bf16(o[k + 4], o[k + 5]),
            pack_bf16(o[k + 6], o[k + 7]));
      if (u0 == 4) flush(reinterpret_cast<char*>(a.out + orow * kNope + c - 32), kNope * 2);
    } else {
      // 128 bytes a row
#pragma unroll
      for (int k = 0; k < 32; k += 4)
        put(k / 4, __float_as_uint(o[k]), __float_as_uint(o[k + 1]), __float_as_uint(o[k + 2]), __float_as_uint(o[k + 3]));
      flush(reinterpret_cast<char*>(plan.o_part + prow * kNope + c), kNope * 4);
    }
  }
  if (lane < live) {
    if (whole) a.lse[orow + lane] = lse;
    else plan.lse_part[prow + lane] = lse;
  }
}

}  // namespace smla
