// Chunk attention on single SMs: the kernel for few query rows (decode steps, drafted
// tokens), where the cache is read about once and an expanded copy would triple the
// traffic.
//
// Tiles of 64 (token, head) rows; shares of the block line (see smla_chunk.h) spread a
// long context over all SMs.  A CTA expands the packed rows itself: S = Q K^T (64 x 64 x
// 512 a block of 64 positions), O += P V (64 x 448 x 64), K and V from one expanded block in
// shared memory.
//
// What bounds it: the chain that each block goes through, not one unit.  64 positions are 37 KB
// of the cache, 1,630 cycles at the copy rate with all SMs reading.  The products take 2,350
// (32 of 64 x 64 x 16 at their measured minimum of 45 cycles; the value product runs at half
// of the tensor rate with 64 rows: 900), the expansion about 1,600 of the integer pipe, the
// softmax about 800.  Expansion, scores, softmax and value product of a block follow one
// another, and the scores and O fill tensor memory, so two blocks in two buffers overlap in
// part only: about 5,100 cycles a block.  32 single tokens of 64 heads over 8,192 positions
// take 77 us (153 MB: 2.0 TB/s, 29 % of the copy rate; tensor pipe 40 % busy, integer pipe
// 53 %), with plan and merge 87 us; two tokens of 16 heads over 131,072 take 69 and 79 us.
// Measured and not kept: f16 operands (96 us against 93 then), two sets of 8 expanding warps
// (93..105), the next block's rows read before this one's expansion (110: spills), through
// shared memory (92 against 85: past the carve-out step) or half a row earlier (87), one lane
// polling for its warp (107).
//
// Expansion without conversions: an e4m3 byte's exponent and mantissa, shifted into bf16's
// fields, are its value times 2^-120 (subnormals included), and one bf16 product by
// 2^(scale byte - 7) puts both powers right, exactly.  The shifts act on four bytes at
// once: the integer pipe is the expansion's bound.  Rows with NaN or with scale bytes past
// 134 take a slower path.
//
// Warps of a CTA: 0..7 softmax and results (64 rows lie in 16 tensor-memory lanes of each
// quarter, which two warps share by columns), 8..23 expand, 24 issues the scores, 25 the
// value products, 26 loads Q.  Every wait is bounded.
#include <cstring>
#include <mutex>

#include "smla_chunk.h"
#include "smla_chunk_rows.cuh"
#include "smla_ptx.cuh"

namespace smla {
namespace {

constexpr int kSoftWarps = 8;              // two for each quarter of tensor memory
constexpr int kExpandWarp0 = 8;
constexpr int kExpandWarps = 16;
constexpr int kRows = 64 / kExpandWarps;   // of a block, a warp
constexpr int kMmaWarp = 24;
constexpr int kPvWarp = 25;
constexpr int kQWarp = 26;
constexpr int kThreads = 28 * 32;
// Registers (setmaxnreg): what the launch gives is split among the warpgroups.
constexpr int kLaunchRegs = 72;
constexpr int kRegsSoft = 80, kRegsExpand = 72, kRegsMma = 56;
static_assert(kRegsSoft * 256 + kRegsExpand * 512 + kRegsMma * 128 <= kLaunchRegs * kThreads, "register split");
static_assert(kRegsSoft >= kLaunchRegs && kRegsExpand >= kLaunchRegs && kRegsMma <= kLaunchRegs,
              "the direction that each role's setmaxnreg takes");
constexpr int kSlab = 64 * 128;            // 64 columns of 64 rows
constexpr int kBuf = 8 * kSlab;            // an expanded block
constexpr int kQOff = 0;
constexpr int kBufOff = 8 * kSlab;
// P of a block takes the place of its rope, which the scores are done with; the buffer is
// filled again only after the value product.  Without 8 KB for P the CTA stays below the
// 196 KB step of the shared-memory carve-out, which leaves the loads 60 KB of L1, not 28 (93 ->
// 85 us).
constexpr int kPOff = kBufOff + 7 * kSlab;     // + kBuf for the second buffer
constexpr int kBarOff = kBufOff + 2 * kBuf;
constexpr int kMaskOff = kBarOff + 256;    // [2 buffers][mapped, not finite][16 half bytes]
constexpr int kMaxOff = kMaskOff + 64;      // float [2 blocks][2 halves][64 rows]: largest scores; later sums
constexpr int kSmem = kMaxOff + 1024 + 1024;
static_assert(kSmem <= 195 * 1024, "the carve-out step, less what the system takes");
constexpr uint32_t kColS = 448;

// FULL / EMPTY: half of a block buffer (columns 0..255, the rest) filled / its value product
// done, two buffers; QFULL / QEMPTY: Q loaded / its last scores done; SFULL / SEMPTY: scores
// in tensor memory / taken by the softmax; PFULL: weights written (one for each buffer: a
// quarter may be a block ahead of another); OEMPTY: results taken.
enum Bar : int { FULL = 0, EMPTY = 4, PFULL = 8, QFULL = 10, QEMPTY, SFULL, SEMPTY, OEMPTY, kBars };

// A row of the blocks on the line, walked tile by tile and each tile's share from its last
// block to its first (scores that a distance bias shapes then fall along the way, and the
// running maximum seldom rises): page and row in it follow by subtractions, divided out at a
// tile's start only.
struct Cursor {
  int x, x1, t, next;     // next: where tile t ends
  int b, left;            // sequence, and its positions from the row's on
  int page, off;
  __device__ __forceinline__ void load(const ChunkPlan& p, int row, int page_size) {
    const int4 tile = p.tile[t];
    next = p.cum[t + 1];
    b = tile.x;
    const int pos = (tile.w + (min(x1, next) - 1 - p.cum[t])) * kChunkBlk + row;
    left = p.seq_len[b] - pos;
    page = pos / page_size;
    off = pos - page * page_size;
  }
  // pages, rest: 64 / page_size and 64 % page_size
  __device__ __forceinline__ void step(const ChunkPlan& p, int row, int page_size, int pages, int rest) {
    ++x;
    if (x == next && x < x1) {
      ++t;
      load(p, row, page_size);
      return;
    }
    left += kChunkBlk;
    page -= pages;
    off -= rest;
    if (off < 0) {
      off += page_size;
      --page;
    }
  }
};

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Four e4m3 bytes -> four bf16, times m.  High bytes: sign and the exponent's upper three
// bits; low bytes: its last bit and the mantissa.
__device__ __forceinline__ uint2 expand4(uint32_t w, uint32_t m) {
  const uint32_t high = (w & 0x80808080u) | ((w >> 4) & 0x07070707u);
  const uint32_t low = (w << 4) & 0xf0f0f0f0u;
  return make_uint2(mul_bf16x2(prmt(low, high, 0x5140), m), mul_bf16x2(prmt(low, high, 0x7362), m));
}
__device__ __forceinline__ uint4 expand8(uint2 w, uint32_t m) {
  const uint2 a = expand4(w.x, m), b = expand4(w.y, m);
  return make_uint4(a.x, a.y, b.x, b.y);
}
// Bits 15 and 31: an infinite or NaN bf16.
__device__ __forceinline__ uint32_t rope_bits(uint32_t w) { return (w & 0x7f807f80u) + 0x00800080u; }
// Any e4m3 NaN among four bytes: a byte of 0x7f carries into its bit 7.
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
__device__ __forceinline__ void sts(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void sts4(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// Predicated forms, so that lanes with and without a word do not part ways.
__device__ __forceinline__ void sts_if(bool p, uint32_t addr, uint4 v) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t@q st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n\t}\n" ::"r"(addr),
               "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(p ? 1 : 0)
               : "memory");
}
__device__ __forceinline__ void sts8_if(bool p, uint32_t addr, uint2 v) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %3, 0;\n\t@q st.shared.v2.u32 [%0], {%1,%2};\n\t}\n" ::"r"(addr), "r"(v.x),
               "r"(v.y), "r"(p ? 1 : 0)
               : "memory");
}
// 8 bytes of the pool (read-only here, once).
__device__ __forceinline__ uint2 ldg_once(const uint8_t* src) {
  uint2 v;
  asm("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(src));
  return v;
}

// The 8-byte words of its warp's rows that a lane l holds.  Words 0..55 of a row are the nope
// part (word w: columns 8 (w % 8) .. + 7 of group w / 8), 56 the scales, 57..72 the rope.
// a[j], b[j]: words l and l + 32 of row j; c[k]: word 64 + l % 9 of row 3 k + l / 9.
constexpr int kTails = (kRows + 2) / 3;
struct RowWords {
  uint2 a[kRows], b[kRows], c[kTails];
};

// Two rows a thread: the 16 rows of a quarter with 32 of their 64 scores of a block, as the
// 16-lane tensor-memory load deals them out: lane 4 g + q has columns 8 j + 2 q and + 1 (of
// the warp's half) of rows g (v[4 j], v[4 j + 1]) and g + 8 (v[4 j + 2], v[4 j + 3]).  Sums
// stay per thread until the end; the maximum is the row's, of both halves.
template <bool MODS>
struct TwoRows {
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, lr[2] = {0.f, 0.f};
  int lo[2] = {0, 0}, hi[2] = {0, 0}, pos[2] = {0, 0};
  float slope2[2] = {0.f, 0.f};
  ScoreMods mods;

  __device__ __forceinline__ TwoRows(const ChunkArgs& a, const ChunkPlan& plan, const int4& tile, int row0)
      : mods(a) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = row0 + 8 * i;
      if (row >= tile.z) continue;
      const int tok = (tile.y + row) / a.H;
      visible(a, tile.x, tok, plan.seq_len[tile.x], &lo[i], &hi[i], &pos[i]);
      if (MODS && a.slopes != nullptr) slope2[i] = a.slopes[tile.y + row - tok * a.H] * kLog2e;
    }
  }

  // The two rows side by side, and half of the columns a warp: the weights are on the way
  // from scores to value product.  most: this block's [2 halves][64 rows] of shared memory.
  __device__ __forceinline__ void weights(float (&v)[16], int s0, const ulonglong2& rows, volatile float* most,
                                          uint32_t (&p)[8], float (&alpha)[2]) {
    const int half = threadIdx.x >> 7, quarter = (threadIdx.x >> 5) & 3, g = (threadIdx.x >> 2) & 7;
    const int col = 32 * half + 2 * (threadIdx.x & 3);
    const float scale2 = mods.scale2;
    if constexpr (MODS) {
      const float from0 = static_cast<float>(pos[0] - s0 - col), from1 = static_cast<float>(pos[1] - s0 - col);
      mods(v, [&](int k) {
        const float c = static_cast<float>(8 * (k / 4) + k % 2);
        return k % 4 < 2 ? make_float2(slope2[0], from0 - c) : make_float2(slope2[1], from1 - c);
      });
    }
    const unsigned long long seen0 = seen_of(rows.x, s0, lo[0], hi[0]), seen1 = seen_of(rows.x, s0, lo[1], hi[1]);
    if (__any_sync(0xffffffffu, (seen0 & seen1) != ~0ull)) {
      const uint32_t at0 = static_cast<uint32_t>(seen0 >> col), at1 = static_cast<uint32_t>(seen1 >> col);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (!((at0 >> (8 * j + e)) & 1)) v[4 * j + e] = -INFINITY;
          if (!((at1 >> (8 * j + e)) & 1)) v[4 * j + 2 + e] = -INFINITY;
        }
    }
    float t[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int j = 1; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] = fmaxf(t[e], v[4 * j + e]);
    float top[2] = {fmaxf(t[0], t[1]), fmaxf(t[2], t[3])}, shift[2];
#pragma unroll
    for (int x = 1; x <= 2; x *= 2) {
      const float u0 = __shfl_xor_sync(0xffffffffu, top[0], x), u1 = __shfl_xor_sync(0xffffffffu, top[1], x);
      top[0] = fmaxf(top[0], u0);
      top[1] = fmaxf(top[1], u1);
    }
    // the other half's maximum (the quarter's two warps meet)
    const int row = 16 * quarter + g;
    if ((threadIdx.x & 3) == 0) {
      most[64 * half + row] = top[0];
      most[64 * half + row + 8] = top[1];
    }
    asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
    top[0] = fmaxf(top[0], most[64 * (half ^ 1) + row]);
    top[1] = fmaxf(top[1], most[64 * (half ^ 1) + row + 8]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (!MODS) top[i] *= scale2;
      const bool raise = top[i] > m[i] + kHeadroom || (m[i] == -INFINITY && top[i] > m[i]);
      alpha[i] = raise ? exp2_fast(m[i] - top[i]) : 1.f;      // 0 while m is -inf
      m[i] = raise ? top[i] : m[i];
      shift[i] = m[i] == -INFINITY ? 0.f : m[i];
    }
    float sum[4] = {0.f, 0.f, 0.f, 0.f}, rsum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float e[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x = v[4 * j + k];
        e[k] = exp2_fast(MODS ? x - shift[k / 2] : fmaf(x, scale2, -shift[k / 2]));
        sum[k] += e[k];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        p[2 * j + i] = pack_bf16(e[2 * i], e[2 * i + 1]);
        rsum[2 * i] += __uint_as_float(p[2 * j + i] << 16);
        rsum[2 * i + 1] += __uint_as_float(p[2 * j + i] & 0xffff0000u);
      }
    }
    // a row of the cache that is not finite is held as zeros; who sees it becomes NaN
    const bool odd0 = (seen0 & rows.y) != 0, odd1 = (seen1 & rows.y) != 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool odd = i == 0 ? odd0 : odd1;
      l[i] = odd ? __uint_as_float(0x7fffffffu) : fmaf(l[i], alpha[i], sum[2 * i] + sum[2 * i + 1]);
      lr[i] = odd ? __uint_as_float(0x7fffffffu) : fmaf(lr[i], alpha[i], rsum[2 * i] + rsum[2 * i + 1]);
    }
  }
};

// Half of the columns of rows row and row + 8 of the tile, as the 16-lane load deals them
// out: final (`whole`), or partial into `slot`.  Four lanes write 32 consecutive bytes of a
// partial row (16 of a final one).
__device__ __forceinline__ void store_result(const ChunkArgs& a, const ChunkPlan& plan, const float (&inv)[2],
                                             const float (&lse)[2], uint32_t tO, const int4& tile, int row,
                                             bool whole, int slot, int half) {
  const int q = threadIdx.x & 3;
  const int64_t orow = static_cast<int64_t>(tile.y) + row, prow = static_cast<int64_t>(slot) * kSingleRows + row;
#pragma unroll 1
  for (int c = 224 * half; c < 224 * half + 224; c += 32) {
    float o[16];
    tmem_ld_16x32(tO + c, o);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (row + 8 * i >= tile.z) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = o[4 * j + 2 * i] * inv[i], y = o[4 * j + 2 * i + 1] * inv[i];
        const int col = c + 8 * j + 2 * q;
        if (whole) *reinterpret_cast<uint32_t*>(a.out + (orow + 8 * i) * kNope + col) = pack_bf16(x, y);
        else *reinterpret_cast<float2*>(plan.o_part + (prow + 8 * i) * kNope + col) = make_float2(x, y);
      }
    }
  }
  if (half == 0 && q == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (row + 8 * i >= tile.z) continue;
      if (whole) a.lse[orow + 8 * i] = lse[i];
      else plan.lse_part[prow + 8 * i] = lse[i];
    }
  }
}

// x[0] of lane 4 g for row g < 8, x[1] for row g + 8, to lane = row.
__device__ __forceinline__ float to_row(const float (&x)[2]) {
  const int src = (threadIdx.x & 7) * 4;
  const float a = __shfl_sync(0xffffffffu, x[0], src), b = __shfl_sync(0xffffffffu, x[1], src);
  return (threadIdx.x & 8) ? b : a;
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// The low halves of 16 bytes side by side.
__device__ __forceinline__ unsigned long long halves(unsigned long long low, unsigned long long high) {
  auto eight = [](unsigned long long x) {
    x = (x | (x >> 4)) & 0x00ff00ff00ff00ffull;
    x = (x | (x >> 8)) & 0x0000ffff0000ffffull;
    return (x | (x >> 16)) & 0x00000000ffffffffull;
  };
  return eight(low) | (eight(high) << 32);
}
// After a wait has run out: products in flight end within microseconds, 1 ms before they lose
// their memory.
__device__ __forceinline__ void drain() {
  const long long t0 = clock64();
  while (clock64() - t0 < 2000000) {
  }
}
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
      mbar_init(bar(i), i < EMPTY ? kExpandWarps : i == SEMPTY || i == PFULL || i == PFULL + 1 || i == OEMPTY ? kSoftWarps : 1);
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

  const int t_first = plan.start[worker], x0 = plan.begin[worker], x1 = plan.begin[worker + 1];

  if (warp >= kExpandWarp0 && warp < kMmaWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsExpand) : "memory");
    // ---------------- expand ----------------
    // Rows 4 w .. + 3 of a block are warp w's; lane j's cursor follows row j % 4; the warp
    // reads a row at once, 256 consecutive bytes a load.  All warps expand a block together,
    // since that lies between a value product and the scores of the block after next; the
    // next block's bytes are on their way meanwhile.
    const int w16 = warp - kExpandWarp0;
    const int mine = kRows * w16 + (lane & (kRows - 1));
    const int c_row = lane / 9, c_word = lane % 9;       // of words c
    if (x0 < x1) {
      const int pages_step = kChunkBlk / a.page_size, rest = kChunkBlk % a.page_size;
      const uint32_t stride = static_cast<uint32_t>(a.stride);
      // page id of the cursor's row, -1 = no row there
      auto lookup = [&](const Cursor& c) {
        if (c.x >= c.x1 || c.left <= 0) return -1;
        if (c.page < a.max_pages) return __ldg(a.table + static_cast<int64_t>(c.b) * a.max_pages + c.page);
        atomicCAS(a.status, 0, SMLA_ERR_INDEX_RANGE);
        return -1;
      };
      // the rows' bytes; returns which of them are mapped.  In the place of a row that is not
      // there the pool's first is read: its position is masked, and what it holds does not
      // matter (a row that is not finite is held as zeros).  Rows of a pool that fits the
      // GPU number far below 2^32.
      uint32_t row_now = 0;
      auto fetch = [&](int id, int off, RowWords& d) {
        const long long r = static_cast<long long>(id) * a.page_size + off;
        const bool there = id >= 0 && r < a.num_rows;
        if (id >= 0 && !there) atomicCAS(a.status, 0, SMLA_ERR_INDEX_RANGE);
        const uint32_t have = __ballot_sync(0xffffffffu, there) & ((1u << kRows) - 1u);
        row_now = there ? static_cast<uint32_t>(r) : 0u;
        const uint8_t* base = a.pool + 8 * lane;
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          const uint8_t* src = base + static_cast<uint64_t>(__shfl_sync(0xffffffffu, row_now, j)) * stride;
          d.a[j] = ldg_once(src);
          d.b[j] = ldg_once(src + 256);
        }
#pragma unroll
        for (int k = 0; k < kTails; ++k) {
          const int j = min(3 * k + c_row, kRows - 1);        // lanes with no such row: any
          d.c[k] = ldg_once(a.pool + static_cast<uint64_t>(__shfl_sync(0xffffffffu, row_now, j)) * stride + 512 + 8 * c_word);
        }
        return have;
      };
      Cursor at;                     // the block whose page ids are fetched next
      at.x = x0;
      at.x1 = x1;
      at.t = t_first;
      at.load(plan, mine, a.page_size);
      RowWords d;
      const int count = x1 - x0;
      uint32_t have = fetch(lookup(at), at.off, d);
      at.step(plan, mine, a.page_size, pages_step, rest);
      int id = lookup(at), off = at.off;
      bool ok = true;
      // word b of this lane: nope, scales (lane 24) or rope; how its NaN are found
      const uint32_t mb = lane < 24 ? 0x7f7f7f7fu : lane > 24 ? 0x7f807f80u : 0u;
      const uint32_t ab = lane < 24 ? 0x01010101u : 0x00800080u;
      const uint32_t tb = lane < 24 ? 0x80808080u : 0x80008000u;
      const int sh = 8 * (lane >> 3);
      const uint32_t pick = 0x4040u + 0x0101u * static_cast<uint32_t>(lane >> 3);   // (byte, 0, byte, 0)
      const uint32_t pick_b = lane < 24 ? pick : 0x4444u;
      const uint32_t dst_nope = sbase + kBufOff + (lane >> 3) * kSlab;
      for (int n = 0; n < count; ++n) {
        const int B = n & 1;
        // 2^(s - 7) as two bf16 of this lane's groups (s: their scale bytes) of each row; lanes
        // 24 .. 31 have no second group
        auto power = [](uint32_t twice) { return twice * 128u + 0x3c003c00u; };
        uint32_t ma[kRows], mx[kRows];
        // anything that the fast path does not cover: NaN, infinite rope values, scale bytes
        // past 134
        uint32_t na = 0, nb = 0, nc = 0, top = 0;
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          na |= nan_bits(d.a[j].x) | nan_bits(d.a[j].y);
          nb |= ((d.b[j].x & mb) + ab) | ((d.b[j].y & mb) + ab);
          const uint32_t sa = prmt(__shfl_sync(0xffffffffu, d.b[j].x, 24), 0, pick);
          const uint32_t sb = prmt(__shfl_sync(0xffffffffu, d.b[j].y, 24), 0, pick_b);
          top = max(top, max(sa, sb));
          ma[j] = power(sa);
          mx[j] = power(sb);
        }
#pragma unroll
        for (int k = 0; k < kTails; ++k) nc |= rope_bits(d.c[k].x) | rope_bits(d.c[k].y);
        const bool odd = (na & 0x80808080u) | (nb & tb) | (nc & 0x80008000u) | (top > 0x00860086u ? 1u : 0u);
        const bool usual = !__any_sync(0xffffffffu, odd);
        uint32_t dropped = 0;        // rows that are not finite: held as zeros
        // The unusual path reads its rows again, one by one: kept in registers for it, they
        // would make the usual path spill.
        auto again = [&](int j, int byte) {      // 8 bytes of row j
          return ldg_once(a.pool + static_cast<uint64_t>(__shfl_sync(0xffffffffu, row_now, j)) * stride + byte);
        };
        if (!usual) {
#pragma unroll 1
          for (int j = 0; j < kRows; ++j) {
            const uint2 wa = again(j, 8 * lane), wb = again(j, 256 + 8 * lane), wc = again(j, 512 + 8 * min(lane, 8));
            const uint32_t sx = __shfl_sync(0xffffffffu, wb.x, 24), sy = __shfl_sync(0xffffffffu, wb.y, 24);
            // a NaN (a scale byte of 255 makes NaN), or past bf16's largest value: seen in the results
            const uint4 oa = expand8_any(wa, (sx >> sh) & 0xffu);
            const uint4 ob = lane < 24 ? expand8_any(wb, (sy >> sh) & 0xffu)
                                       : lane > 24 ? make_uint4(wb.x, wb.y, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t bad = rope_bits(oa.x) | rope_bits(oa.y) | rope_bits(oa.z) | rope_bits(oa.w) | rope_bits(ob.x) |
                                 rope_bits(ob.y) | rope_bits(ob.z) | rope_bits(ob.w) | rope_bits(wc.x) | rope_bits(wc.y);
            dropped |= __any_sync(0xffffffffu, (bad & 0x80008000u) != 0) ? 1u << j : 0u;
          }
        }
        const uint32_t parity = ((n >> 1) - 1) & 1;
        if (n >= 2) ok = warp_wait(bar(EMPTY + 2 * B), parity, stop, a.status);
        if (!ok) break;
        const uint32_t dn = dst_nope + kRows * w16 * 128 + B * kBuf;
        const int r7 = (kRows * w16) & 7;                 // the warp's first row modulo 8
        auto unit = [&](int j) { return j * 128 + (((lane & 7) ^ (r7 + j)) << 4); };    // the lane's unit of row j
        if (usual) {
          // two rows at a time, their conversions interleaved; times 2^(s - 7) as two bf16
#pragma unroll
          for (int j0 = 0; j0 < kRows; j0 += 2) {
            uint4 o[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
              o[j] = expand8(d.a[j0 + j], ma[j0 + j]);
#pragma unroll
            for (int j = 0; j < 2; ++j) sts(dn + unit(j0 + j), o[j]);
          }
        } else {
#pragma unroll 1
          for (int j = 0; j < kRows; ++j) {
            const uint2 wa = again(j, 8 * lane);
            const uint32_t s = (again(j, kNope).x >> sh) & 0xffu;
            sts(dn + unit(j), (dropped >> j) & 1 ? make_uint4(0u, 0u, 0u, 0u) : expand8_any(wa, s));
          }
        }
        if (lane == 0) {
          masks[B * 32 + w16] = static_cast<uint8_t>(have);
          masks[B * 32 + 16 + w16] = static_cast<uint8_t>(dropped);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && !(n == a.fault_block && w16 == 0)) mbar_arrive(bar(FULL + 2 * B));
        if (n >= 2) ok = warp_wait(bar(EMPTY + 2 * B + 1), parity, stop, a.status);
        if (!ok) break;
        // the rope: word w of row j
        const uint32_t dr = sbase + kBufOff + 7 * kSlab + kRows * w16 * 128 + B * kBuf;
        auto rope = [&](int j, int w) { return dr + j * 128 + (((w >> 1) ^ (r7 + j)) << 4) + 8 * (w & 1); };
        if (usual) {
#pragma unroll
          for (int j0 = 0; j0 < kRows; j0 += 2) {
            uint4 o[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
              o[j] = expand8(d.b[j0 + j], mx[j0 + j]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              sts_if(lane < 24, dn + 4 * kSlab + unit(j0 + j), o[j]);
              sts8_if(lane > 24, rope(j0 + j, (lane - 25) & 15), d.b[j0 + j]);
            }
          }
        } else {
#pragma unroll 1
          for (int j = 0; j < kRows; ++j) {
            const uint2 wb = again(j, 256 + 8 * lane);
            const uint32_t s = (again(j, kNope).y >> sh) & 0xffu;
            const bool drop = (dropped >> j) & 1;
            sts_if(lane < 24, dn + 4 * kSlab + unit(j), drop ? make_uint4(0u, 0u, 0u, 0u) : expand8_any(wb, s));
            sts8_if(lane > 24, rope(j, (lane - 25) & 15), drop ? make_uint2(0u, 0u) : wb);
          }
        }
#pragma unroll
        for (int k = 0; k < kTails; ++k) {
          const int j = 3 * k + c_row;
          sts8_if(j < kRows && lane < 27, rope(j & (kRows - 1), 7 + c_word), (dropped >> j) & 1 ? make_uint2(0u, 0u) : d.c[k]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(FULL + 2 * B + 1));
        // the next block's bytes, and the page ids of the one after it
        have = fetch(id, off, d);
        at.step(plan, mine, a.page_size, pages_step, rest);
        id = lookup(at);
        off = at.off;
      }
    }
  } else if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsMma) : "memory");
    // The whole warp walks its schedule, one elected lane issues (descriptors stay uniform).
    // Two warps, so that a value product that is ready does not wait for a block that is
    // not, nor the other way round.
    const uint64_t d0 = smem_desc(sbase, 16, 1024, SWZ_128B), dv = smem_desc(sbase, kSlab, 1024, SWZ_128B);
    const uint32_t hi = static_cast<uint32_t>(d0 >> 32);
    if (warp == kMmaWarp) {
      // ---------------- scores ----------------
      constexpr uint32_t kIdQK = idesc_bf16(64, 64, false, false);
      const uint32_t lq = static_cast<uint32_t>(d0), lk = lq + (kBufOff >> 4);
      uint32_t n = 0, k = 0;               // blocks and tiles so far
      bool ok = true;
      for (int x = x0, t = t_first; ok && x < x1; ++t, ++k) {
        const int end = min(x1, plan.cum[t + 1]);
        ok = warp_wait(bar(QFULL), k & 1, stop, a.status);
        for (; ok && x < end; ++x, ++n) {
          if (n > 0) ok = warp_wait(bar(SEMPTY), (n - 1) & 1, stop, a.status);
          for (int h = 0; ok && h < 2; ++h) {
            ok = warp_wait(bar(FULL + 2 * (n & 1) + h), (n >> 1) & 1, stop, a.status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t la = lq + h * ((4 * kSlab) >> 4), lb = lk + (n & 1) * (kBuf >> 4) + h * ((4 * kSlab) >> 4);
            if (elect_one()) {
#pragma unroll 1
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  mma_f16_ss_hl(tmem + kColS, la + ((c * kSlab + i * 32) >> 4), hi, lb + ((c * kSlab + i * 32) >> 4), hi,
                                kIdQK, c + i > 0 ? 1u : static_cast<uint32_t>(h));
              if (h == 1) {
                mma_commit(bar(SFULL));
                if (x + 1 == end) mma_commit(bar(QEMPTY));
              }
            }
            __syncwarp();
          }
        }
      }
      if (!ok) drain();
    } else if (warp == kPvWarp) {
      // ---------------- value products ----------------
      constexpr uint32_t kIdV0 = idesc_bf16(64, 256, false, true), kIdV1 = idesc_bf16(64, 192, false, true);
      const uint32_t lp = static_cast<uint32_t>(d0) + (kPOff >> 4), lv = static_cast<uint32_t>(dv) + (kBufOff >> 4);
      uint32_t n = 0, k = 0;
      bool ok = true;
      for (int x = x0, t = t_first; ok && x < x1; ++t, ++k) {
        const int end = min(x1, plan.cum[t + 1]);
        uint32_t old = 0;                  // the tile's first product overwrites O
        for (; ok && x < end; ++x, ++n, old = 1) {
          ok = warp_wait(bar(PFULL + (n & 1)), (n >> 1) & 1, stop, a.status);
          if (ok && old == 0 && k > 0) ok = warp_wait(bar(OEMPTY), (k - 1) & 1, stop, a.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t lb = lv + (n & 1) * (kBuf >> 4);
          if (elect_one()) {
            // columns 0..255 first: the next block's may be written while 256..447 follow
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_f16_ss_hl(tmem, lp + (n & 1) * (kBuf >> 4) + ((i * 32) >> 4), hi, lb + ((i * 2048) >> 4), hi, kIdV0, i > 0 ? 1u : old);
            mma_commit(bar(EMPTY + 2 * (n & 1)));
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_f16_ss_hl(tmem + 256, lp + (n & 1) * (kBuf >> 4) + ((i * 32) >> 4), hi, lb + ((4 * kSlab + i * 2048) >> 4), hi, kIdV1,
                            i > 0 ? 1u : old);
            mma_commit(bar(EMPTY + 2 * (n & 1) + 1));
          }
          __syncwarp();
        }
      }
      if (!ok) drain();
    } else if (warp == kQWarp) {
      // ---------------- Q ----------------
      bool ok = true;
      uint32_t k = 0;
      for (int x = x0, t = t_first; ok && x < x1; ++t, ++k) {
        if (k > 0) ok = warp_wait(bar(QEMPTY), (k - 1) & 1, stop, a.status);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(bar(QFULL), 8 * kSlab);
          for (int c = 0; c < 8; ++c)
            tma_load_2d(sbase + kQOff + c * kSlab, &qmap, 64 * c, plan.tile[t].y, bar(QFULL));
        }
        __syncwarp();
        x = min(x1, plan.cum[t + 1]);
      }
      // the last copy has landed before the CTA may end
      if (k > 0) warp_wait(bar(QFULL), (k - 1) & 1, stop, a.status);
    }
  } else if (warp < kExpandWarp0) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft) : "memory");
    // ---------------- softmax and results ----------------
    // Warps w and w + 4: rows 16 w .. + 15, columns 0..31 and 32..63 of a block; two rows and
    // 8 of their scores a thread for the weights, lane = row for O, of which each warp has
    // half of the columns.
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + kColS + 32 * half + lanes, tO = tmem + lanes;
    const int g = lane >> 2;
    volatile float* most = reinterpret_cast<volatile float*>(smem + kMaxOff);
    // P: rows 16 quarter + g and + 8 (the same row modulo 8), columns 2 (lane % 4) .. of unit j
    const uint32_t p0 = sbase + kPOff + (16 * quarter + g) * 128 + 4 * (lane & 3), p1 = p0 + 8 * 128;
    uint32_t n = 0;
    int x = x0, t = t_first, i = 0, held = 0;
    bool ok = true;
    for (; ok && x < x1; ++t) {
      const int4 tile = plan.tile[t];
      const int begin = plan.cum[t], after = plan.cum[t + 1], end = min(x1, after);
      const int nb = end - x, blk = tile.w + (end - 1 - begin);     // the first block
      // rows past the tile stay whatever they are (a product's rows do not mix), so a warp
      // without rows only keeps step
      TwoRows<MODS> st(a, plan, tile, 16 * quarter + g);
      const bool idle = 16 * quarter >= tile.z;
      for (i = 0; ok && i < nb; ++i, ++n) {
        ok = warp_wait(bar(FULL + 2 * (n & 1)), (n >> 1) & 1, stop, a.status);     // the masks' writers
        if (!ok) break;
        const volatile unsigned long long* mk =
            reinterpret_cast<const volatile unsigned long long*>(smem + kMaskOff + (n & 1) * 32);
        const unsigned long long m0 = mk[0], m1 = mk[1], d0 = mk[2], d1 = mk[3];
        ulonglong2 rows = make_ulonglong2(~0ull, 0ull);
        if (__any_sync(0xffffffffu, (m0 & m1) != 0x0f0f0f0f0f0f0f0full || (d0 | d1) != 0))
          rows = make_ulonglong2(halves(m0, m1), halves(d0, d1));
        ok = warp_wait(bar(SFULL), n & 1, stop, a.status);
        if (!ok) break;
        if (idle) {
          if (lane == 0) {
            mbar_arrive(bar(SEMPTY));
            mbar_arrive(bar(PFULL + (n & 1)));
          }
          continue;
        }
        tc_fence_after();
        float v[16];
        tmem_ld_16x32(tS, v);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(SEMPTY));
        uint32_t p[8];
        float alpha[2];
        st.weights(v, (blk - i) * kChunkBlk, rows, most + (n & 1) * 128, p, alpha);
        // O may be rescaled once the value product before this one is done
        if (i > 0 && __any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
          ok = warp_wait(bar(EMPTY + 2 * ((n - 1) & 1) + 1), ((n - 1) >> 1) & 1, stop, a.status);
          if (!ok) {
            held = 1;
            break;
          }
          tc_fence_after();
          const float f = to_row(alpha);
          rescale_rows(tO, lane < 16 ? f : 1.f, 224 * half, 224);
        }
        const uint32_t pb = (n & 1) * kBuf;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sts4(p0 + pb + (((j + 4 * half) ^ g) << 4), p[2 * j]);
          sts4(p1 + pb + (((j + 4 * half) ^ g) << 4), p[2 * j + 1]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(PFULL + (n & 1)));
      }
      if (!ok) break;
      ok = warp_wait(bar(EMPTY + 2 * ((n - 1) & 1) + 1), ((n - 1) >> 1) & 1, stop, a.status);
      if (!ok) break;
      tc_fence_after();
      if (!idle) {
        // the sums of both halves, through the maxima's places (their readers of the last
        // blocks are done: each warp's arrivals for P came after its reads)
        float l[2], lr[2], inv[2], lse[2];
        asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          l[i] = quad_sum(st.l[i]);
          lr[i] = quad_sum(st.lr[i]);
          if ((lane & 3) == 0) {
            most[64 * half + 16 * quarter + g + 8 * i] = l[i];
            most[128 + 64 * half + 16 * quarter + g + 8 * i] = lr[i];
          }
        }
        asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // in the same order in both warps
          const float o = most[64 * (half ^ 1) + 16 * quarter + g + 8 * i], orr = most[128 + 64 * (half ^ 1) + 16 * quarter + g + 8 * i];
          const float ls = half == 0 ? l[i] + o : o + l[i], lrs = half == 0 ? lr[i] + orr : orr + lr[i];
          inv[i] = inverse_sum(ls, lrs);
          lse[i] = lse_of(st.m[i], ls);
        }
        asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");     // read before the next tile's maxima
        store_result(a, plan, inv, lse, tO, tile, 16 * quarter + g, begin >= x0 && after <= x1,
                     2 * worker + (begin < x0 ? 0 : 1), half);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(OEMPTY));
      x = end;
    }
    // A wait has run out.  The quarter's other warp may have come further: both hold all
    // meetings of the schedule, one a block and three a tile, so that neither waits for good.
    if (!ok)
      for (; x < x1; ++t, i = 0, held = 0) {
        const int end = min(x1, plan.cum[t + 1]);
        if (16 * quarter < plan.tile[t].z)
          for (int k = end - x + 3 - i - held; k > 0; --k) asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
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
      // the register split assumes the launch's share: a build that differs is refused,
      // since its increase would never be granted
      cudaFuncAttributes fa;
      e = cudaFuncGetAttributes(&fa, single_kernel<MODS>);
      if (e != cudaSuccess) return e;
      if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidKernelImage;
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
