// Chunk attention on single SMs: the kernel for few query rows (decode steps, drafted
// tokens), where the cache is read about once and an expanded copy would triple the
// traffic.
//
// Tiles of 64 (token, head) rows; shares of the block line (see smla_chunk.h) spread a
// long context over all SMs.  A CTA expands the packed rows itself: S = Q K^T (64 x 64 x
// 512 a block of 64 positions), O += P V (64 x 448 x 64), K and V from one expanded block in
// shared memory.
//
// What bounds it.  64 positions are 37 KB of the cache: 1,630 cycles at the measured
// bandwidth with all SMs reading.  The products take at least 45 cycles each at 64 x 64 x 16
// (measured; 32 of them) and half of the tensor rate at 64 rows (900 cycles for the value
// product): about 2,350 cycles a block.  Shared memory moves 64 KB of Q, 64 KB of K, 72 KB
// of V and P and 64 KB of expanded rows, 2,060 cycles.  So a block of one or two SMs' worth
// of rows is bound by the tensor core at small tiles, within 1.5 of the cache's bandwidth.
//
// Expansion without conversions: an e4m3 byte's exponent and mantissa, shifted into bf16's
// fields, are its value times 2^-120 (subnormals included), and one bf16 product by
// 2^(scale byte - 7) puts both powers right, exactly.  Rows with NaN or with scale bytes
// past 134 take a slower path.
//
// Warps of a CTA: 0..3 softmax and results (lanes 0..15: 64 rows lie in 16 tensor-memory
// lanes of each quarter), 4..11 expand (8 rows of each block; the next block's bytes are in
// flight in registers, the one after next's page ids too), 12 loads Q and issues the
// products.  Every wait is bounded.
#include <cstring>
#include <mutex>

#include "smla_chunk.h"
#include "smla_chunk_rows.cuh"
#include "smla_ptx.cuh"

namespace smla {
namespace {

constexpr int kExpandWarp0 = 4;
constexpr int kExpandWarps = 8;
constexpr int kMmaWarp = 12;
constexpr int kThreads = 13 * 32;
constexpr int kSlab = 64 * 128;            // 64 columns of 64 rows
constexpr int kBuf = 8 * kSlab;            // an expanded block
constexpr int kQOff = 0;
constexpr int kBufOff = 8 * kSlab;
constexpr int kPOff = kBufOff + 2 * kBuf;
constexpr int kBarOff = kPOff + kSlab;
constexpr int kMaskOff = kBarOff + 256;    // mapped and poisoned positions: [2 buffers][2][8 bytes]
constexpr int kSmem = kMaskOff + 64 + 1024;
constexpr uint32_t kColS = 448;

// FULL / EMPTY: block buffer filled / its value product done; QFULL / QEMPTY: Q loaded /
// its last scores done; SFULL / SEMPTY: scores in tensor memory / taken by the softmax;
// PFULL: weights written; PV: value product done; OEMPTY: results taken.
enum Bar : int { FULL = 0, EMPTY = 2, QFULL = 4, QEMPTY, SFULL, SEMPTY, PFULL, PV, OEMPTY, kBars };

// A position on the line, walked block by block.
struct Cursor {
  int x, x1, t, next;     // next: where tile t ends
  int b, blk, len;
  __device__ __forceinline__ void load(const ChunkPlan& p) {
    const int4 tile = p.tile[t];
    next = p.cum[t + 1];
    b = tile.x;
    blk = tile.w + (x - p.cum[t]);
    len = p.seq_len[b];
  }
  __device__ __forceinline__ void step(const ChunkPlan& p) {
    ++x;
    ++blk;
    if (x < x1 && x == next) {
      ++t;
      load(p);
    }
  }
};

// Two e4m3 bytes (in bits 8..15 and 24..31) as bf16 times 2^-120, times m.
__device__ __forceinline__ uint32_t expand2(uint32_t t, uint32_t m) {
  const uint32_t v = (t & 0x80008000u) | ((t >> 4) & 0x07f007f0u);
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(m));
  return r;
}
__device__ __forceinline__ uint32_t spread(uint32_t w, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(w), "r"(sel));
  return r;
}
__device__ __forceinline__ uint4 expand8(uint2 w, uint32_t m) {
  return make_uint4(expand2(spread(w.x, 0x1404), m), expand2(spread(w.x, 0x3424), m),
                    expand2(spread(w.y, 0x1404), m), expand2(spread(w.y, 0x3424), m));
}
// Any e4m3 NaN among four bytes.
__device__ __forceinline__ uint32_t nan_bits(uint32_t w) { return (w & 0x7f7f7f7fu) + 0x01010101u; }

// 8 bytes with any scale byte, in 32 bits; out of line: unusual rows only.
__device__ __noinline__ uint4 expand8_any(uint2 w, uint32_t s) {
  const float sc = __uint_as_float(s == 0u ? 0x00400000u : (s == 255u ? 0x7fffffffu : (s << 23)));
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t two = ((i < 2 ? w.x : w.y) >> (16 * (i & 1))) & 0xffffu;
    uint32_t h2;
    const uint16_t in = static_cast<uint16_t>(two);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(in));
    float lo, hi;
    asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;}" : "=f"(lo), "=f"(hi) : "r"(h2));
    o[i] = pack_bf16(lo * sc, hi * sc);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ bool not_finite(uint32_t v) {
  return (v & 0x7f80u) == 0x7f80u || (v & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ void sts(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint2 ldg_once(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// The bytes of one row that a lane holds: lane q of a row's 8 has words q + 8 g of the nope
// part (columns 64 g + 8 q .. + 7 of group g), the scale word, and 16 bytes of the rope.
struct RowBytes {
  uint2 w[7], sc, r0, r1;
};

template <bool MODS>
__global__ void __launch_bounds__(kThreads, 1)
    single_kernel(const ChunkArgs a, const ChunkPlan plan, const __grid_constant__ CUtensorMap qmap) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int worker = blockIdx.x;
  auto bar = [&](int i) { return sbase + kBarOff + 8u * static_cast<uint32_t>(i); };
  volatile uint32_t* taddr = reinterpret_cast<volatile uint32_t*>(smem + kBarOff + 8 * kBars);
  volatile int* stop = reinterpret_cast<volatile int*>(smem + kBarOff + 8 * kBars + 8);
  volatile uint8_t* masks = smem + kMaskOff;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBars; ++i)
      mbar_init(bar(i), i < EMPTY ? kExpandWarps : i == SEMPTY || i == PFULL || i == OEMPTY ? 4 : 1);
    *stop = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(sbase + kBarOff + 8 * kBars, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *taddr;
  grid_dep_wait();
  grid_dep_launch();

  const int total = plan.head[1], per = plan.head[2], tiles = plan.head[0];
  const int x0 = min(static_cast<long long>(total), static_cast<long long>(worker) * per);
  const int x1 = min(total, x0 + per);
  const int t_first = x0 < x1 ? find_last_le(plan.cum, tiles + 1, x0) : 0;

  if (warp >= kExpandWarp0 && warp < kMmaWarp) {
    // ---------------- expand ----------------
    const int w8 = warp - kExpandWarp0, q = lane & 7;
    const int row0 = 8 * w8 + (lane >> 3);          // and row0 + 4
    if (x0 < x1) {
      // page ids of the two rows of the cursor's block: -1 = no row there
      auto pages = [&](const Cursor& c, int (&id)[2]) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int s = c.blk * kChunkBlk + row0 + 4 * j;
          id[j] = -1;
          if (c.x < c.x1 && s < c.len) {
            const int page = s / a.page_size;
            if (page < a.max_pages) id[j] = __ldg(a.table + static_cast<int64_t>(c.b) * a.max_pages + page);
            else if (q == 0) atomicCAS(a.status, 0, SMLA_ERR_INDEX_RANGE);
          }
        }
      };
      // the bytes of those rows; have: bit j set where row j is mapped
      auto fetch = [&](const Cursor& c, const int (&id)[2], RowBytes (&d)[2], uint32_t& have) {
        have = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          long long row = -1;
          if (id[j] >= 0) {
            const int s = c.blk * kChunkBlk + row0 + 4 * j;
            row = static_cast<long long>(id[j]) * a.page_size + s % a.page_size;
            if (row >= a.num_rows) {
              row = -1;
              if (q == 0) atomicCAS(a.status, 0, SMLA_ERR_INDEX_RANGE);
            }
          }
          if (row >= 0) {
            have |= 1u << j;
            const uint8_t* src = a.pool + row * a.stride;
#pragma unroll
            for (int g = 0; g < 7; ++g) d[j].w[g] = ldg_once(src + 64 * g + 8 * q);
            d[j].sc = ldg_once(src + kNope);
            d[j].r0 = ldg_once(src + 456 + 16 * q);
            d[j].r1 = ldg_once(src + 456 + 16 * q + 8);
          } else {
#pragma unroll
            for (int g = 0; g < 7; ++g) d[j].w[g] = make_uint2(0u, 0u);
            d[j].sc = make_uint2(0x7f7f7f7fu, 0x007f7f7fu);
            d[j].r0 = d[j].r1 = make_uint2(0u, 0u);
          }
        }
      };
      Cursor at;                     // the block whose page ids are fetched next
      at.x = x0;
      at.x1 = x1;
      at.t = t_first;
      at.load(plan);
      Cursor c1 = at;                // the block whose bytes are fetched next
      int id[2];
      RowBytes cur[2], nxt[2];
      uint32_t have, have_next = 0;
      pages(at, id);
      fetch(c1, id, cur, have);
      at.step(plan);
      c1 = at;
      pages(at, id);
      bool ok = true;
      for (int n = 0; ok && n < x1 - x0; ++n) {
        fetch(c1, id, nxt, have_next);
        at.step(plan);
        c1 = at;
        pages(at, id);
        const int buf = n & 1;
        if (n >= 2) ok = warp_wait(bar(EMPTY + buf), ((n >> 1) - 1) & 1, stop, a.status);
        if (!ok) break;
        uint32_t poison = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const RowBytes& d = cur[j];
          const int row = row0 + 4 * j;
          const uint32_t dst = sbase + kBufOff + buf * kBuf + row * 128 + ((q ^ (row & 7)) << 4);
          uint32_t odd = 0;
#pragma unroll
          for (int g = 0; g < 7; ++g) odd |= nan_bits(d.w[g].x) | nan_bits(d.w[g].y);
          odd &= 0x80808080u;
          // scale bytes past 134: + 121 carries into bit 8 of a 16-bit lane
          odd |= (((d.sc.x & 0x00ff00ffu) + 0x00790079u) | (((d.sc.x >> 8) & 0x00ff00ffu) + 0x00790079u) |
                  ((d.sc.y & 0x00ff00ffu) + 0x00790079u) | (((d.sc.y >> 8) & 0x000000ffu) + 0x00000079u)) & 0x01000100u;
          odd |= (not_finite(d.r0.x) | not_finite(d.r0.y) | not_finite(d.r1.x) | not_finite(d.r1.y)) ? 1u : 0u;
          if (__any_sync(0xffffffffu, odd != 0)) {
            uint4 o[8];
            bool bad = false;
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              o[g] = g < 7 ? expand8_any(d.w[g], ((g < 4 ? d.sc.x : d.sc.y) >> (8 * (g & 3))) & 0xffu)
                           : make_uint4(d.r0.x, d.r0.y, d.r1.x, d.r1.y);
              bad |= not_finite(o[g].x) | not_finite(o[g].y) | not_finite(o[g].z) | not_finite(o[g].w);
            }
            // the 8 lanes of a row agree: zeros for a row that is not finite
            const bool drop = (__ballot_sync(0xffffffffu, bad) >> (lane & 24)) & 0xffu;
            poison |= drop ? 1u << j : 0u;
#pragma unroll
            for (int g = 0; g < 8; ++g) sts(dst + g * kSlab, drop ? make_uint4(0u, 0u, 0u, 0u) : o[g]);
          } else {
#pragma unroll
            for (int g = 0; g < 7; ++g) {
              // 2^(s - 7) as two bf16
              const uint32_t s = ((g < 4 ? d.sc.x : d.sc.y) >> (8 * (g & 3))) & 0xffu;
              sts(dst + g * kSlab, expand8(d.w[g], ((s + 120u) << 7) * 0x00010001u));
            }
            sts(dst + 7 * kSlab, make_uint4(d.r0.x, d.r0.y, d.r1.x, d.r1.y));
          }
        }
        // row 8 w8 + i (i < 4): lane 8 i, bit 0; i >= 4: lane 8 (i - 4), bit 1
        const uint32_t m0 = __ballot_sync(0xffffffffu, have & 1), m1 = __ballot_sync(0xffffffffu, have & 2);
        const uint32_t p0 = __ballot_sync(0xffffffffu, poison & 1), p1 = __ballot_sync(0xffffffffu, poison & 2);
        if (lane == 0) {
          auto pick = [](uint32_t lo, uint32_t hi) {
            uint32_t v = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) v |= ((lo >> (8 * i)) & 1u) << i | ((hi >> (8 * i)) & 1u) << (4 + i);
            return static_cast<uint8_t>(v);
          };
          masks[buf * 16 + w8] = pick(m0, m1);
          masks[buf * 16 + 8 + w8] = pick(p0, p1);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(FULL + buf));
#pragma unroll
        for (int j = 0; j < 2; ++j) cur[j] = nxt[j];
        have = have_next;
      }
    }
  } else if (warp == kMmaWarp) {
    // ---------------- Q and products ----------------
    // The whole warp walks the schedule, one elected lane issues (descriptors stay uniform).
    constexpr uint32_t kIdQK = idesc_bf16(64, 64, false, false);
    constexpr uint32_t kIdV0 = idesc_bf16(64, 256, false, true);
    constexpr uint32_t kIdV1 = idesc_bf16(64, 192, false, true);
    const uint64_t d0 = smem_desc(sbase, 16, 1024, SWZ_128B), dv = smem_desc(sbase, kSlab, 1024, SWZ_128B);
    const uint32_t hi = static_cast<uint32_t>(d0 >> 32);
    const uint32_t lq = static_cast<uint32_t>(d0), lk = lq + (kBufOff >> 4), lp = lq + (kPOff >> 4);
    const uint32_t lv = static_cast<uint32_t>(dv) + (kBufOff >> 4);
    uint32_t n = 0, nv = 0, nq = 0;      // scores, value products and tiles so far
    bool ok = true;
    for (int x = x0, t = t_first; ok && x < x1; ++t) {
      const int end = min(x1, plan.cum[t + 1]);
      const int nb = end - x;
      const int row0 = plan.tile[t].y;
      if (nq > 0) ok = warp_wait(bar(QEMPTY), (nq - 1) & 1, stop, a.status);
      if (!ok) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(bar(QFULL), 8 * kSlab);
        for (int c = 0; c < 8; ++c) tma_load_2d(sbase + kQOff + c * kSlab, &qmap, 64 * c, row0, bar(QFULL));
      }
      __syncwarp();
      ok = warp_wait(bar(QFULL), nq & 1, stop, a.status);
      for (int i = 0; ok && i <= nb; ++i) {
        if (i < nb) {
          ok = warp_wait(bar(FULL + (n & 1)), (n >> 1) & 1, stop, a.status);
          if (ok && n > 0) ok = warp_wait(bar(SEMPTY), (n - 1) & 1, stop, a.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t lb = lk + (n & 1) * (kBuf >> 4);
          if (elect_one()) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_f16_ss_hl(tmem + kColS, lq + ((c * kSlab + k * 32) >> 4), hi, lb + ((c * kSlab + k * 32) >> 4), hi,
                              kIdQK, c + k > 0 ? 1u : 0u);
            mma_commit(bar(SFULL));
            if (i == nb - 1) mma_commit(bar(QEMPTY));
          }
          __syncwarp();
          ++n;
        }
        if (i > 0) {
          ok = warp_wait(bar(PFULL), nv & 1, stop, a.status);
          if (ok && i == 1 && nq > 0) ok = warp_wait(bar(OEMPTY), (nq - 1) & 1, stop, a.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t lb = lv + (nv & 1) * (kBuf >> 4);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t acc = k > 0 ? 1u : (i > 1 ? 1u : 0u);
              mma_f16_ss_hl(tmem, lp + ((k * 32) >> 4), hi, lb + ((k * 2048) >> 4), hi, kIdV0, acc);
              mma_f16_ss_hl(tmem + 256, lp + ((k * 32) >> 4), hi, lb + ((4 * kSlab + k * 2048) >> 4), hi, kIdV1, acc);
            }
            mma_commit(bar(EMPTY + (nv & 1)));
            mma_commit(bar(PV));
          }
          __syncwarp();
          ++nv;
        }
      }
      ++nq;
      x = end;
    }
    if (!ok) {   // copies and products in flight end within microseconds: 1 ms before they lose their memory
      const long long t0 = clock64();
      while (clock64() - t0 < 2000000) {
      }
    }
  } else if (warp < kExpandWarp0) {
    // ---------------- softmax and results: lane < 16 = row 16 warp + lane ----------------
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tS = tmem + kColS + lanes, tO = tmem + lanes;
    const int row = 16 * warp + (lane & 15);
    uint32_t n = 0;
    bool ok = true;
    for (int x = x0, t = t_first; ok && x < x1; ++t) {
      const int4 tile = plan.tile[t];
      const int begin = plan.cum[t], after = plan.cum[t + 1], end = min(x1, after);
      const int nb = end - x, blk = tile.w + (x - begin);
      const bool mine = lane < 16 && row < tile.z;
      // lanes 16..31 follow lanes 0..15 on scores of no row; rows past the tile stay whatever
      // they are (a product's rows do not mix), so a warp without rows only keeps step
      RowState<MODS> st(a, plan, tile, row, row < tile.z);
      const bool idle = 16 * warp >= tile.z;
      for (int i = 0; ok && i < nb; ++i, ++n) {
        ok = warp_wait(bar(SFULL), n & 1, stop, a.status);
        if (ok) ok = warp_wait(bar(FULL + (n & 1)), (n >> 1) & 1, stop, a.status);   // the masks' writers
        if (!ok) break;
        if (idle) {
          if (lane == 0) mbar_arrive(bar(SEMPTY));
          if (i > 0) ok = warp_wait(bar(PV), (n - 1) & 1, stop, a.status);
          if (!ok) break;
          if (lane == 0) mbar_arrive(bar(PFULL));
          continue;
        }
        tc_fence_after();
        float v[64];
        tmem_ld32(tS, v);
        tmem_ld32(tS + 32, v + 32);
        const volatile unsigned long long* mk =
            reinterpret_cast<const volatile unsigned long long*>(smem + kMaskOff + (n & 1) * 16);
        const ulonglong2 rows = make_ulonglong2(mk[0], mk[1]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(SEMPTY));
        uint32_t p[32];
        const float shrink = st.weights(v, (blk + i) * kChunkBlk, rows, p);
        const float alpha = lane < 16 ? shrink : 1.f;
        if (i > 0) {
          ok = warp_wait(bar(PV), (n - 1) & 1, stop, a.status);
          if (!ok) break;
          tc_fence_after();
          rescale_rows(tO, alpha);
        }
        if (lane < 16) store_weights(sbase + kPOff, row, p);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(PFULL));
      }
      if (!ok) break;
      ok = warp_wait(bar(PV), (n - 1) & 1, stop, a.status);
      if (!ok) break;
      tc_fence_after();
      store_rows<kSingleRows>(a, plan, st, tO, tile, row, mine, begin >= x0 && after <= x1,
                              2 * worker + (begin < x0 ? 0 : 1));
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(OEMPTY));
      x = end;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

std::mutex g_mu;

template <bool MODS>
cudaError_t launch(const ChunkArgs& a, const ChunkPlan& p, int workers, cudaStream_t stream) {
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    if (!done[dev]) {
      e = cudaFuncSetAttribute(single_kernel<MODS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
  }
  CUtensorMap qmap;
  std::memset(static_cast<void*>(&qmap), 0, sizeof(qmap));
  e = encode_rows(&qmap, a.q, static_cast<int64_t>(a.T) * a.H, kSingleRows);
  if (e != cudaSuccess) return e;
  return launch_programmatic(single_kernel<MODS>, dim3(workers), dim3(kThreads), kSmem, stream, a, p, qmap);
}

}  // namespace

cudaError_t launch_chunk_single(const ChunkArgs& a, const ChunkPlan& p, int workers, cudaStream_t stream) {
  return a.cap > 0.f || a.slopes != nullptr ? launch<true>(a, p, workers, stream)
                                            : launch<false>(a, p, workers, stream);
}

}  // namespace smla
