// Chunk attention on single SMs: the kernel for few query rows (decode steps, drafted
// tokens), where the cache is read about once and an expanded copy would triple the
// traffic.
//
// Tiles of 64 (token, head) rows; shares of the block line (see smla_chunk.h) spread a
// long context over all SMs.  A CTA expands the packed rows itself: S = Q K^T (64 x 64 x
// 512 a block of 64 positions), O += P V (64 x 448 x 64), K and V from one expanded block in
// shared memory, Q and P from tensor memory.
//
// What bounds it: the chain that each block goes through, not one unit.  64 positions of 8-bit rows are 37 KB of
// the cache, 1,630 cycles at the copy rate with all SMs reading (24 KB and 1,030 of 4-bit rows).  The products take
// 2,000 (32 of 64 x 64 x 16 by way of tensor memory 1,060, the value product 940: 64 rows run at half the tensor
// rate), the expansion about 1,600 of the integer pipe (700 of 4-bit rows), the softmax about 800.  Expansion,
// scores, softmax and value product of a block follow one another, so three blocks are on their way: the scores of
// one beside the expansion of the next and the value product of the one before.  From the release of a block's places
// to that of the same places again are 8,900 cycles: expansion 2,700, scores 2,200 beside the other products, softmax
// 2,100 beside the expanding warps, value product.  32 single tokens of 64 heads over 8,192 positions take 74 us of
// 8-bit rows (153 MB: 2.1 TB/s, 30 % of the copy rate) and 52 of 4-bit rows (tensor pipe 37 % of the time, issue
// slots 52 %, integer pipe 42 % of the active cycles).
// Measured and not kept, two blocks and Q in shared memory: f16 operands (96 us against 93 then), two sets of 8
// expanding warps (93..105), the next block's rows read before this one's expansion (110: spills), through
// shared memory (92 against 85: past the carve-out step) or half a row earlier (87), one lane
// polling for its warp (107).  4-bit rows, three blocks: a block more on its way to registers 65 against 62, one proxy
// fence a block 59 against 57.5, a ring of 7 half blocks past the carve-out step 66 against 55, a set of expanding
// warps for each half of a block 57 against 55.
//
// Expansion without conversions: an e4m3 byte's exponent and mantissa, shifted into bf16's
// fields, are its value times 2^-120 (subnormals included), and one bf16 product by
// 2^(scale byte - 7) puts both powers right, exactly.  The shifts act on four bytes at
// once: the integer pipe is the expansion's bound.  Rows with NaN or with scale bytes past
// 134 take a slower path.  4-bit rows the same way (expand_nibbles); any scale byte, in two products where one
// power of two is not enough.
//
// Warps of a CTA: 0..7 softmax, Q and results (64 rows lie in 16 tensor-memory lanes of each
// quarter, which two warps share by columns), 8..23 expand, 24 issues the scores, 25 the
// value products, 26 makes the plan of few tiles.  Every wait is bounded.
#include <mutex>
#include <type_traits>

#include "smla_chunk.h"
#include "smla_chunk_rows.cuh"
#include "smla_ptx.cuh"

namespace smla {
namespace {

constexpr int kSoftWarps = 8;              // two for each quarter of tensor memory
constexpr int kExpandWarp0 = 8;
constexpr int kExpandWarps = 16;
// Warps that expand a block together.  4-bit rows: two sets of 8 take the blocks in turn, since a warp's way through
// a block (its loads, two waits, two proxy fences) is mostly latency.
template <bool ROW4>
constexpr int kSetWarps = ROW4 ? 8 : kExpandWarps;
constexpr int kMmaWarp = 24;
constexpr int kPvWarp = 25;
constexpr int kPlanWarp = 26;
constexpr int kThreads = 28 * 32;
// Registers (setmaxnreg): what the launch gives is split among the warpgroups.
constexpr int kLaunchRegs = 72;
constexpr int kRegsSoft = 80, kRegsExpand = 72, kRegsMma = 56;
static_assert(kRegsSoft * 256 + kRegsExpand * 512 + kRegsMma * 128 <= kLaunchRegs * kThreads, "register split");
static_assert(kRegsSoft >= kLaunchRegs && kRegsExpand >= kLaunchRegs && kRegsMma <= kLaunchRegs,
              "the direction that each role's setmaxnreg takes");
constexpr int kSlab = 64 * 128;            // 64 columns of 64 rows
constexpr int kHalf = 4 * kSlab;           // columns 0..255 or 256..511 of an expanded block
// Half blocks are expanded into a ring of places, a block's two one after the other: three blocks, so that
// expansion, scores and value product need not wait for one another's ends.  With Q in tensor memory the CTA
// stays below the 196 KB step of the shared-memory carve-out, which leaves the loads 60 KB of L1, not 28.
constexpr int kPlaces = 6;
constexpr int kBarOff = kPlaces * kHalf;
constexpr int kMasks = 3;                  // blocks whose masks are held: a block is expanded again only after its weights
constexpr int kMaskOff = kBarOff + 192;    // [3 blocks][mapped, not finite][16 half bytes]
constexpr int kMaxOff = kMaskOff + 96;     // float [2 blocks][2 halves][64 rows]: largest scores; later sums
// The plan of few tiles: int4 [tiles] sequence + 256 rows, first row, positions of the sequence, first block;
// int [tiles + 1] where each begins on the line; the share's begin, end and first tile.
constexpr int kPlanOff = kMaxOff + 1024, kPlanCum = kPlanOff + 16 * kFewTiles, kPlanShare = kPlanCum + 4 * (kFewTiles + 1);
constexpr int kSmem = kPlanShare + 12 + 1024;
static_assert(kSmem <= 195 * 1024, "the carve-out step, less what the system takes");

// Tensor memory.  64 rows of a product lie in 16 lanes of each quarter, the lower ones or the upper, so
// that 512 columns hold twice as much.  Lower: Q (two bf16 a column), the scores of two blocks, columns 384..447 of
// O, the weights of two blocks (two bf16 a column).  Upper: columns 0..383 of O, and the weights once more.  (A
// product's first operand lies in the lanes of its result.)  Weights by way of shared memory, with its fence, took
// 54.8 us against 53.0 (32 single tokens, 4-bit rows; 79.4 and 78.4 of 8-bit rows).
constexpr uint32_t kColS = 256, kColTail = 384, kColP = 448, kUpper = 16u << 16;
__device__ __forceinline__ uint32_t o_column(uint32_t tmem, int c) {
  return tmem + static_cast<uint32_t>(c) + (c < static_cast<int>(kColTail) ? kUpper : 0u);
}

// FULL / EMPTY: a place of the ring filled / its value product done; PFULL: weights in tensor memory, two blocks in
// turn (a quarter may be a block ahead of another, and no more, since the third one's weights wait for the value
// product that the other holds up); QFULL: a tile's Q in tensor memory; SFULL /
// SEMPTY: scores of a block in tensor memory / taken by the softmax, two in turn; OEMPTY: results taken.
enum Bar : int {
  FULL = 0, EMPTY = kPlaces, PFULL = 2 * kPlaces, QFULL = PFULL + 2, SFULL, SEMPTY = SFULL + 2, OEMPTY = SEMPTY + 2, kBars
};

// A place of the ring, and the parity of its uses.
struct Place {
  uint32_t at = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == kPlaces) {
      at = 0;
      phase ^= 1;
    }
  }
  // of half block i (without a state to keep: registers of the softmax)
  static __device__ __forceinline__ Place of(uint32_t i) {
    Place p;
    const uint32_t use = i / kPlaces;
    p.at = i - use * kPlaces;
    p.phase = use & 1;
    return p;
  }
};

__device__ __forceinline__ int lds4(uint32_t addr) {
  int v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ int4 lds16(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// The plan as a worker reads it: worked out from a tile's number, in shared memory, or in the workspace.
template <bool EVEN>
struct Plan {
  const ChunkArgs& a;
  const ChunkPlan& p;
  uint32_t smem;
  __device__ __forceinline__ bool few() const { return !is_even<EVEN>(p) && p.few; }
  // a worker's share and its first tile
  __device__ __forceinline__ int begin(int w) const { return few() ? lds4(smem + kPlanShare) : plan_begin<EVEN>(p, w); }
  __device__ __forceinline__ int end(int w) const { return few() ? lds4(smem + kPlanShare + 4) : plan_begin<EVEN>(p, w + 1); }
  __device__ __forceinline__ int start(int w, int x) const {
    return few() ? lds4(smem + kPlanShare + 8) : plan_start<EVEN>(p, w, x);
  }
  __device__ __forceinline__ int cum(int t) const { return few() ? lds4(smem + kPlanCum + 4 * t) : plan_cum<EVEN>(p, t); }
  // sequence, first row, rows, first block
  __device__ __forceinline__ int4 tile(int t) const {
    if (!few()) return plan_tile<EVEN>(p, t);
    const int4 v = lds16(smem + kPlanOff + 16 * t);
    return make_int4(v.x & 255, v.y, v.x >> 8, v.w);
  }
  // positions of tile t's sequence b
  __device__ __forceinline__ int len(int t, int b) const {
    return few() ? lds4(smem + kPlanOff + 16 * t + 8) : plan_len<EVEN>(a, p, b);
  }
};

// A row of the blocks on the line, walked tile by tile and each tile's share from its last
// block to its first (scores that a distance bias shapes then fall along the way, and the
// running maximum seldom rises): page and row in it follow by subtractions, divided out at a
// tile's start only.
struct Cursor {
  int x, x1, t, next;     // next: where tile t ends
  int b, left;            // sequence, and its positions from the row's on
  int page, off;
  template <bool EVEN>
  __device__ __forceinline__ void load(const Plan<EVEN>& p, int row, int page_size) {
    const int4 tile = p.tile(t);
    next = p.cum(t + 1);
    b = tile.x;
    const int pos = (tile.w + (min(x1, next) - 1 - p.cum(t))) * kChunkBlk + row;
    left = p.len(t, b) - pos;
    page = pos / page_size;
    off = pos - page * page_size;
  }
  // pages, rest: 64 / page_size and 64 % page_size
  template <bool EVEN>
  __device__ __forceinline__ void step(const Plan<EVEN>& p, int row, int page_size, int pages, int rest) {
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
// The largest magnitudes (signs aside; NaN wins).
__device__ __forceinline__ uint32_t largest_bf16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t largest_of(const uint4& v) {
  return largest_bf16(largest_bf16(v.x, v.y), largest_bf16(v.z, v.w));
}
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
// The store of 16 lanes x 16 columns: lane 4 g + q of the warp gives columns 4 j + q of lanes g (v[2 j]) and g + 8.
__device__ __forceinline__ void tmem_st_16x16(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
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
constexpr int kRows8 = 64 / kSetWarps<false>, kTails = (kRows8 + 2) / 3;
struct RowWords {
  uint2 a[kRows8], b[kRows8], c[kTails];
};

// 4-bit rows: lane l holds the 16-byte words 4 k + l / 8 (w[k]; k = 5 of lanes 24 .. 31: word 22 once more) of
// row l % 8 of its warp.  Words 0..13 of a row are 32 nope columns each, one scale group; 14 is the
// scales, 15..22 the rope.
struct RowWords4 {
  uint4 w[6];
};
__device__ __forceinline__ uint4 ldg16_once(const uint8_t* src) {
  uint4 v;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(src));
  return v;
}
// Eight e2m1 nibbles (column 2 p in nibble p, 2 p + 1 in nibble p + 4) -> eight bf16.  A nibble's
// sign at bit 15 and its exponent and mantissa at bits 8..6 are its value times 2^-126, subnormals
// included, and one product by 2^(scale byte - 1) (m) puts both powers right, exactly.
__device__ __forceinline__ uint4 expand_nibbles(uint32_t w, uint32_t m) {
  constexpr uint32_t kSign = 0x80008000u, kMag = 0x01c001c0u;
  return make_uint4(mul_bf16x2(((w << 12) & kSign) | ((w << 6) & kMag), m),
                    mul_bf16x2(((w << 8) & kSign) | ((w << 2) & kMag), m),
                    mul_bf16x2(((w << 4) & kSign) | ((w >> 2) & kMag), m),
                    mul_bf16x2((w & kSign) | ((w >> 6) & kMag), m));
}
__device__ __forceinline__ uint4 mul4(uint4 v, uint32_t m) {
  return make_uint4(mul_bf16x2(v.x, m), mul_bf16x2(v.y, m), mul_bf16x2(v.z, m), mul_bf16x2(v.w, m));
}
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
// Nibbles that times 2^(s - 127) pass bf16's largest value, or a scale byte of 255.
__device__ __forceinline__ bool past_bf16(const uint4& v, uint32_t s) {
  const uint32_t w = s == 254 ? v.x | v.y | v.z | v.w : 0u;                          // 2 and above
  const uint32_t u = s == 253 ? (v.x & (v.x << 1)) | (v.y & (v.y << 1)) | (v.z & (v.z << 1)) | (v.w & (v.w << 1)) : 0u;
  return s == 255 || ((w | u) & 0x44444444u) != 0;                                   // 4 and 6
}

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

  __device__ __forceinline__ TwoRows(const ChunkArgs& a, const int4& tile, int len, int row0)
      : mods(a) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = row0 + 8 * i;
      if (row >= tile.z) continue;
      const int tok = (tile.y + row) / a.H;
      visible(a, tile.x, tok, len, &lo[i], &hi[i], &pos[i]);
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
    // two scores, weights or sums an instruction: the columns of a row side by side
    Two sum[2] = {Two(0.f), Two(0.f)}, rsum[2] = {Two(0.f), Two(0.f)};
    const Two by(MODS ? 1.f : scale2);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const Two x(v[4 * j + 2 * i], v[4 * j + 2 * i + 1]), away(-shift[i]);
        float e0, e1;
        (MODS ? x + away : fma2(x, by, away)).get(&e0, &e1);
        e0 = exp2_fast(e0);
        e1 = exp2_fast(e1);
        sum[i] = sum[i] + Two(e0, e1);
        p[2 * j + i] = pack_bf16(e0, e1);
        rsum[i] = rsum[i] + Two(__uint_as_float(p[2 * j + i] << 16), __uint_as_float(p[2 * j + i] & 0xffff0000u));
      }
    // a row of the cache that is not finite is held as zeros; who sees it becomes NaN
    const bool odd0 = (seen0 & rows.y) != 0, odd1 = (seen1 & rows.y) != 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool odd = i == 0 ? odd0 : odd1;
      float s0, s1, r0, r1;
      sum[i].get(&s0, &s1);
      rsum[i].get(&r0, &r1);
      l[i] = odd ? __uint_as_float(0x7fffffffu) : fmaf(l[i], alpha[i], s0 + s1);
      lr[i] = odd ? __uint_as_float(0x7fffffffu) : fmaf(lr[i], alpha[i], r0 + r1);
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
    tmem_ld_16x32(o_column(tO, c), o);
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

// A warp's half of the columns of O, times alpha of its two rows; seldom, so out of line.
__device__ __noinline__ void rescale_half(uint32_t tO, float alpha0, float alpha1, int half) {
#pragma unroll 1
  for (int c = 224 * half; c < 224 * half + 224; c += 32) {
    float o[16];
    tmem_ld_16x32(o_column(tO, c), o);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] *= k % 4 < 2 ? alpha0 : alpha1;
    tmem_st_16x32(o_column(tO, c), o);
  }
  tmem_wait_st();
}

// A warp's half of the columns of its 16 rows of the tile's Q into tensor memory, as the 16-lane store takes them:
// lane 4 g + q has columns (pairs of bf16) 8 j + 2 q and + 1 of rows g and g + 8.  Rows past the tile are zeros.
__device__ __forceinline__ void load_q(const ChunkArgs& a, const int4& tile, uint32_t tQ, int quarter, int half) {
  const int lane = threadIdx.x & 31, row = 16 * quarter + (lane >> 2);
  const uint16_t* src = a.q + (static_cast<int64_t>(tile.y) + row) * kQkDim + 256 * half + 4 * (lane & 3);
  const bool in0 = row < tile.z, in1 = row + 8 < tile.z;
#pragma unroll 2
  for (int c = 0; c < 4; ++c) {
    float r[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint2 none = make_uint2(0u, 0u);
      const uint2 u = in0 ? __ldg(reinterpret_cast<const uint2*>(src + 64 * c + 16 * j)) : none;
      const uint2 v = in1 ? __ldg(reinterpret_cast<const uint2*>(src + 8 * kQkDim + 64 * c + 16 * j)) : none;
      r[4 * j] = __uint_as_float(u.x);
      r[4 * j + 1] = __uint_as_float(u.y);
      r[4 * j + 2] = __uint_as_float(v.x);
      r[4 * j + 3] = __uint_as_float(v.y);
    }
    tmem_st_16x32(tQ + 128 * half + 32 * c, r);
  }
  tmem_wait_st();
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

// The plan of 32 sequences and tiles at most, by one warp: what make_plan does, a lane a sequence and then a lane a
// tile.  Every CTA needs its own share; the first one leaves the cut tiles for the merge.
__device__ __forceinline__ int lanes_before(int v, int* total) {
  const int lane = threadIdx.x & 31;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  *total = __shfl_sync(0xffffffffu, s, 31);
  return s - v;
}
__device__ __forceinline__ void plan_few(const ChunkArgs& a, const ChunkPlan& p, uint32_t smem, int worker) {
  const int lane = threadIdx.x & 31, workers = gridDim.x;
  const Sequence s = sequence(a, lane);        // nothing past the last
  int tiles, blocks;
  const int t0 = lanes_before((s.n * a.H + kSingleRows - 1) / kSingleRows, &tiles);
  const int b0 = lanes_before(s.blocks, &blocks);      // 32 * 2^25 at most
  const int held = seq_len(p, s, b0);
  bool report = held != s.len && lane < a.B;
  if (__any_sync(0xffffffffu, s.wrong)) {
    tiles = 0;
    report = true;
  }
  int b = 0;
  for (int i = 0; i < a.B; ++i)
    if (__shfl_sync(0xffffffffu, t0, i) <= lane) b = i;
  const int first = __shfl_sync(0xffffffffu, s.first, b), last = first + __shfl_sync(0xffffffffu, s.n, b);
  const int len = __shfl_sync(0xffffffffu, held, b), base = __shfl_sync(0xffffffffu, t0, b);
  int row = 0, rows = 0, blk = 0, n = 0;
  if (lane < tiles) {
    row = first * a.H + (lane - base) * kSingleRows;
    rows = min(kSingleRows, last * a.H - row);
    tile_blocks(a, b, row, rows, len, &blk, &n);
  }
  int line;
  const int at = lanes_before(n, &line);       // 2^30 at most
  if (report && worker == 0) atomicCAS(a.status, 0, SMLA_ERR_INDEX_RANGE);
  auto put = [&](uint32_t to, int v) { sts4(smem + to, static_cast<uint32_t>(v)); };
  if (lane < tiles) {
    sts(smem + kPlanOff + 16 * lane, make_uint4(static_cast<uint32_t>(b | rows << 8), static_cast<uint32_t>(row),
                                                static_cast<uint32_t>(len), static_cast<uint32_t>(blk)));
    put(kPlanCum + 4 * lane, at);
  }
  if (lane == 0) put(kPlanCum + 4 * tiles, line);
  __syncwarp();
  const int per = max(kMinShare, (line + workers - 1) / workers), snap = min(kSnap, per / 4);
  auto cum = [&](int t) { return lds4(smem + kPlanCum + 4 * t); };
  // where share c begins, and the tile there (-1 behind the line)
  auto border = [&](int c, int* t) {
    int x = min(c * per, line);                // 152 * (2^30 / 152 + 2) at most
    *t = -1;
    if (x == line) return x;
    int lo = 0;
    for (int hi = tiles; hi - lo > 1;) {
      const int mid = (lo + hi) >> 1;
      if (cum(mid) <= x) lo = mid;
      else hi = mid;
    }
    if (x - cum(lo) <= snap) x = cum(lo);
    else if (cum(lo + 1) - x <= snap) x = cum(++lo);
    if (x < line) *t = lo;
    return x;
  };
  if (lane < 2) {
    int t;
    const int x = border(worker + lane, &t);
    put(kPlanShare + 4 * lane, x);
    if (lane == 0) put(kPlanShare + 8, t);
  }
  if (worker != 0) return;
  // tiles that a border lies inside: the last shares that begin at the tile's start or before, and before its end
  int c0 = 0, c1 = 0;
  if (lane < tiles) {
    auto share = [&](int x) {
      int t, c = min(x / per, workers - 1);
      while (c > 0 && border(c, &t) > x) --c;
      while (c + 1 < workers && border(c + 1, &t) <= x) ++c;
      return c;
    };
    c0 = share(at);
    c1 = share(at + n - 1);
  }
  const uint32_t cuts = __ballot_sync(0xffffffffu, c0 != c1);
  if (c0 != c1) p.cut[__popc(cuts & ((1u << lane) - 1))] = make_int4(row, rows, c0, c1);
  if (lane == 0) p.head[2] = __popc(cuts);
}

template <bool MODS, bool ROW4>
__global__ void __launch_bounds__(kThreads, 1)
    single_kernel(const ChunkArgs a, const ChunkPlan plan) {
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
      mbar_init(bar(i), i < EMPTY ? kSetWarps<ROW4> : i < PFULL || i == SFULL || i == SFULL + 1 ? 1 : kSoftWarps);
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

  constexpr bool EVEN = ROW4 && !MODS;     // may be a sparse call
  const Plan<EVEN> line = {a, plan, sbase};
  if (line.few()) {
    if (warp == kPlanWarp) plan_few(a, plan, sbase, worker);
    __syncthreads();
  }
  const int x0 = line.begin(worker), x1 = line.end(worker), t_first = line.start(worker, x0);

  if (warp >= kExpandWarp0 && warp < kMmaWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsExpand) : "memory");
    // ---------------- expand ----------------
    // Rows kRows w .. of a block are warp w's of a set; lane j's cursor follows row j % kRows.  8-bit rows: all
    // 16 warps expand a block together, and a warp reads a row at once, 256 consecutive bytes a load.  4-bit
    // rows: two sets of 8 warps take the blocks in turn, and a load is 64 bytes of each of a warp's 8 rows.  The
    // next block's bytes are on their way meanwhile.
    constexpr int kRows = 64 / kSetWarps<ROW4>, kSets = kExpandWarps / kSetWarps<ROW4>;      // kRows: of a block, a warp
    const int w16 = (warp - kExpandWarp0) % kSetWarps<ROW4>, set = kSets > 1 ? (warp - kExpandWarp0) / kSetWarps<ROW4> : 0;
    const int mine = kRows * w16 + (lane & (kRows - 1));
    const int c_row = lane / 9, c_word = lane % 9;       // of words c
    if (x0 + set < x1) {
      const int pages_step = kChunkBlk / a.page_size, rest = kChunkBlk % a.page_size;
      const uint32_t stride = static_cast<uint32_t>(a.stride);
      // page id of the cursor's row, -1 = no row there
      auto lookup = [&](const Cursor& c) {
        if (c.x >= c.x1 || c.left <= 0) return -1;
        if (c.page < a.max_pages) {
          const int id = __ldg(a.table + static_cast<int64_t>(c.b) * a.max_pages + c.page);
          if (!ROW4 || a.pages == nullptr || id < 0) return id;
          // a listed position: its page, then its row
          const int page = id / a.listed_page_size;
          if (page < a.max_listed_pages) {
            const int phys = __ldg(a.pages + static_cast<int64_t>(c.b) * a.max_listed_pages + page);
            if (phys < 0) return -1;
            const long long r = static_cast<long long>(phys) * a.listed_page_size + (id - page * a.listed_page_size);
            if (r < a.num_rows) return static_cast<int>(r);
          }
        }
        atomicCAS(a.status, 0, SMLA_ERR_INDEX_RANGE);
        return -1;
      };
      // the rows' bytes; returns which of them are mapped.  In the place of a row that is not
      // there the pool's first is read: its position is masked, and what it holds does not
      // matter (a row that is not finite is held as zeros).  Rows of a pool that fits the
      // GPU number far below 2^32.
      uint32_t row_now = 0;
      auto fetch = [&](int id, int off, auto& d) {
        const long long r = static_cast<long long>(id) * a.page_size + off;
        const bool there = id >= 0 && r < a.num_rows;
        if (id >= 0 && !there) atomicCAS(a.status, 0, SMLA_ERR_INDEX_RANGE);
        const uint32_t have = __ballot_sync(0xffffffffu, there) & ((1u << kRows) - 1u);
        row_now = there ? static_cast<uint32_t>(r) : 0u;
        if constexpr (ROW4) {
          const uint8_t* src = a.pool + static_cast<uint64_t>(row_now) * stride + 16 * (lane >> 3);
#pragma unroll
          for (int k = 0; k < 5; ++k) d.w[k] = ldg16_once(src + 64 * k);
          d.w[5] = ldg16_once(src + (lane < 24 ? 320 : 304));
          return have;
        } else {
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
        }
      };
      Cursor at;                     // the block whose page ids are fetched next
      at.x = x0;
      at.x1 = x1;
      at.t = t_first;
      at.load(line, mine, a.page_size);
      auto advance = [&](int blocks) {
#pragma unroll
        for (int i = 0; i < blocks; ++i) at.step(line, mine, a.page_size, pages_step, rest);
      };
      if (kSets > 1 && set > 0) advance(1);
      std::conditional_t<ROW4, RowWords4, RowWords> d;
      const int count = x1 - x0;
      uint32_t have = fetch(lookup(at), at.off, d);
      advance(kSets);
      int id = lookup(at), off = at.off;
      bool ok = true;
      if constexpr (ROW4) {
        const int j = lane & 7, w = lane >> 3;
        const uint32_t key = static_cast<uint32_t>(j);               // of the swizzle: the row modulo 8
        const uint32_t row = sbase + (kRows * w16 + j) * 128;
        auto unit = [&](uint32_t u) { return (u ^ key) << 4; };
        // 2^(s - 1) as two bf16, in two factors past bf16's exponents
        auto first = [](uint32_t s) { return (min(s, 128u) + 126u) * 0x00800080u; };
        auto second = [](uint32_t s) { return (max(s, 128u) - 1u) * 0x00800080u; };
        for (int n = set; n < count; n += kSets) {
          // the scale bytes of the lane's four nope words (the fourth: words 12 and 13, lanes below 16)
          uint32_t s[4];
          {
            const int from = 16 + j;
            const uint32_t sx = __shfl_sync(0xffffffffu, d.w[3].x, from), sy = __shfl_sync(0xffffffffu, d.w[3].y, from);
            const uint32_t sz = __shfl_sync(0xffffffffu, d.w[3].z, from), sw = __shfl_sync(0xffffffffu, d.w[3].w, from);
            s[0] = (sx >> (8 * w)) & 0xffu;
            s[1] = (sy >> (8 * w)) & 0xffu;
            s[2] = (sz >> (8 * w)) & 0xffu;
            s[3] = w < 2 ? (sw >> (8 * w)) & 0xffu : 0u;
          }
          const uint32_t most_s = max(max(s[0], s[1]), max(s[2], s[3]));
          const bool large = __any_sync(0xffffffffu, most_s > 128u);
          // rows that are not finite are held as zeros
          uint32_t largest = largest_bf16(largest_of(d.w[4]), largest_of(d.w[5]));
          if (w == 3) largest = largest_bf16(largest, largest_of(d.w[3]));
          const bool rope_odd = (rope_bits(largest) & 0x80008000u) != 0;
          uint32_t dropped = 0;
          if (__any_sync(0xffffffffu, rope_odd || most_s >= 253u)) {
            bool bad = rope_odd || (w < 2 && past_bf16(d.w[3], s[3]));
#pragma unroll
            for (int k = 0; k < 3; ++k) bad |= past_bf16(d.w[k], s[k]);
            const uint32_t who = __ballot_sync(0xffffffffu, bad);
            dropped = (who | who >> 8 | who >> 16 | who >> 24) & 0xffu;
            if ((dropped >> j) & 1) {
#pragma unroll
              for (int k = 0; k < 6; ++k) d.w[k] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          // word 4 k + w of the nope part: four 16-byte units of a slab, two words to one
          auto word = [&](const uint4& v, uint32_t scale, uint32_t at) {
            const uint32_t m1 = first(scale), m2 = second(scale);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4 o = expand_nibbles(word_of(v, i), m1);
              if (large) o = mul4(o, m2);
              sts(at + unit(4 * (w & 1) + i), o);
            }
          };
          const Place p0 = Place::of(2 * n), p1 = Place::of(2 * n + 1);
          uint32_t to = row + p0.at * kHalf + (w >> 1) * kSlab;
          if (n >= 3) ok = warp_wait(bar(EMPTY + p0.at), p0.phase ^ 1, stop, a.status);
          if (!ok) break;
          word(d.w[0], s[0], to);
          word(d.w[1], s[1], to + 2 * kSlab);
          if (lane == 0) {
            masks[(n % kMasks) * 32 + w16] = static_cast<uint8_t>(have);
            masks[(n % kMasks) * 32 + 16 + w16] = static_cast<uint8_t>(dropped);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && !(n == a.fault_block && w16 == 0)) mbar_arrive(bar(FULL + p0.at));
          if (n >= 3) ok = warp_wait(bar(EMPTY + p1.at), p1.phase ^ 1, stop, a.status);
          if (!ok) break;
          to = row + p1.at * kHalf + (w >> 1) * kSlab;
          word(d.w[2], s[2], to);
          if (w < 2) word(d.w[3], s[3], to + 2 * kSlab);
          // the rope: its unit 0 is word 15, 1 + w word 16 + w, 5 + w word 20 + w
          const uint32_t rope = row + p1.at * kHalf + 3 * kSlab;
          sts(rope + unit(1 + w), d.w[4]);
          sts(rope + unit(w == 3 ? 0 : 5 + w), w == 3 ? d.w[3] : d.w[5]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(FULL + p1.at));
          have = fetch(id, off, d);
          advance(kSets);
          id = lookup(at);
          off = at.off;
        }
      } else {
        // word b of this lane: nope, scales (lane 24) or rope; how its NaN are found
        const uint32_t mb = lane < 24 ? 0x7f7f7f7fu : lane > 24 ? 0x7f807f80u : 0u;
        const uint32_t ab = lane < 24 ? 0x01010101u : 0x00800080u;
        const uint32_t tb = lane < 24 ? 0x80808080u : 0x80008000u;
        const int sh = 8 * (lane >> 3);
        const uint32_t pick = 0x4040u + 0x0101u * static_cast<uint32_t>(lane >> 3);   // (byte, 0, byte, 0)
        const uint32_t pick_b = lane < 24 ? pick : 0x4444u;
        const uint32_t dst_nope = sbase + (lane >> 3) * kSlab;
        Place place;
        int turn = 0;                  // of the masks' three
        for (int n = 0; n < count; ++n) {
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
          if (n >= 3) ok = warp_wait(bar(EMPTY + place.at), place.phase ^ 1, stop, a.status);
          if (!ok) break;
          uint32_t dn = dst_nope + kRows * w16 * 128 + place.at * kHalf;
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
            masks[turn * 32 + w16] = static_cast<uint8_t>(have);
            masks[turn * 32 + 16 + w16] = static_cast<uint8_t>(dropped);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && !(n == a.fault_block && w16 == 0)) mbar_arrive(bar(FULL + place.at));
          place.next();
          if (n >= 3) ok = warp_wait(bar(EMPTY + place.at), place.phase ^ 1, stop, a.status);
          if (!ok) break;
          dn = dst_nope + kRows * w16 * 128 + place.at * kHalf;
          // the rope: word w of row j
          const uint32_t dr = sbase + 3 * kSlab + kRows * w16 * 128 + place.at * kHalf;
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
                sts_if(lane < 24, dn + unit(j0 + j), o[j]);
                sts8_if(lane > 24, rope(j0 + j, (lane - 25) & 15), d.b[j0 + j]);
              }
            }
          } else {
#pragma unroll 1
            for (int j = 0; j < kRows; ++j) {
              const uint2 wb = again(j, 256 + 8 * lane);
              const uint32_t s = (again(j, kNope).y >> sh) & 0xffu;
              const bool drop = (dropped >> j) & 1;
              sts_if(lane < 24, dn + unit(j), drop ? make_uint4(0u, 0u, 0u, 0u) : expand8_any(wb, s));
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
          if (lane == 0) mbar_arrive(bar(FULL + place.at));
          place.next();
          turn = turn + 1 == kMasks ? 0 : turn + 1;
          // the next block's bytes, and the page ids of the one after it
          have = fetch(id, off, d);
          at.step(line, mine, a.page_size, pages_step, rest);
          id = lookup(at);
          off = at.off;
        }
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
      const uint32_t lk = static_cast<uint32_t>(d0);
      uint32_t n = 0, k = 0;               // blocks and tiles so far
      Place place;
      bool ok = true;
      for (int x = x0, t = t_first; ok && x < x1; ++t, ++k) {
        const int end = min(x1, line.cum(t + 1));
        ok = warp_wait(bar(QFULL), k & 1, stop, a.status);
        for (; ok && x < end; ++x, ++n) {
          if (n >= 2) ok = warp_wait(bar(SEMPTY + (n & 1)), ((n >> 1) - 1) & 1, stop, a.status);
          for (int h = 0; ok && h < 2; ++h) {
            ok = warp_wait(bar(FULL + place.at), place.phase, stop, a.status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t q = tmem + 128 * h, lb = lk + place.at * (kHalf >> 4);
            if (elect_one()) {
#pragma unroll 1
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  mma_f16_ts_hl(tmem + kColS + 64 * (n & 1), q + 32 * c + 8 * i, lb + ((c * kSlab + i * 32) >> 4), hi, kIdQK,
                                c + i > 0 ? 1u : static_cast<uint32_t>(h));
              if (h == 1) mma_commit(bar(SFULL + (n & 1)));
            }
            __syncwarp();
            place.next();
          }
        }
      }
      if (!ok) drain();
    } else if (warp == kPvWarp) {
      // ---------------- value products ----------------
      constexpr uint32_t kId256 = idesc_bf16(64, 256, false, true), kId128 = idesc_bf16(64, 128, false, true),
                         kId64 = idesc_bf16(64, 64, false, true);
      const uint32_t lv = static_cast<uint32_t>(dv);
      uint32_t n = 0, k = 0;               // blocks and tiles so far
      Place place;
      bool ok = true;
      for (int x = x0, t = t_first; ok && x < x1; ++t, ++k) {
        const int end = min(x1, line.cum(t + 1));
        uint32_t old = 0;                  // the tile's first product overwrites O
        for (; ok && x < end; ++x, ++n, old = 1) {
          ok = warp_wait(bar(PFULL + (n & 1)), (n >> 1) & 1, stop, a.status);
          if (ok && old == 0 && k > 0) ok = warp_wait(bar(OEMPTY), (k - 1) & 1, stop, a.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t first = place.at;
          place.next();
          const uint32_t l0 = lv + first * (kHalf >> 4), l1 = lv + place.at * (kHalf >> 4);
          const uint32_t tail = tmem + kColP + 32 * (n & 1), p = tail + kUpper;
          if (elect_one()) {
            // columns 0..255 first: their place may be filled again while 256..447 follow
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_f16_ts_hl(o_column(tmem, 0), p + 8 * i, l0 + ((i * 2048) >> 4), hi, kId256, i > 0 ? 1u : old);
            mma_commit(bar(EMPTY + first));
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_f16_ts_hl(o_column(tmem, 256), p + 8 * i, l1 + ((i * 2048) >> 4), hi, kId128, i > 0 ? 1u : old);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_f16_ts_hl(o_column(tmem, kColTail), tail + 8 * i, l1 + ((2 * kSlab + i * 2048) >> 4), hi, kId64,
                            i > 0 ? 1u : old);
            mma_commit(bar(EMPTY + place.at));
          }
          __syncwarp();
          place.next();
        }
      }
      if (!ok) drain();
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
    auto give_q = [&](int t) {
      load_q(a, line.tile(t), tmem + lanes, quarter, half);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(QFULL));
    };
    const uint32_t tP = tmem + kColP + 16 * half + lanes;
    uint32_t n = 0;
    int x = x0, t = t_first, i = 0, held = 0;
    bool ok = true;
    if (x < x1) give_q(t);
    for (; ok && x < x1; ++t) {
      const int4 tile = line.tile(t);
      const int begin = line.cum(t), after = line.cum(t + 1), end = min(x1, after);
      const int nb = end - x, blk = tile.w + (end - 1 - begin);     // the first block
      // rows past the tile stay whatever they are (a product's rows do not mix), so a warp
      // without rows only keeps step
      TwoRows<MODS> st(a, tile, line.len(t, tile.x), 16 * quarter + g);
      const bool idle = 16 * quarter >= tile.z;
      for (i = 0; ok && i < nb; ++i, ++n) {
        ok = warp_wait(bar(FULL + Place::of(2 * n).at), Place::of(2 * n).phase, stop, a.status);     // the masks' writers
        if (!ok) break;
        const volatile unsigned long long* mk =
            reinterpret_cast<const volatile unsigned long long*>(smem + kMaskOff + (n % kMasks) * 32);
        ulonglong2 rows = make_ulonglong2(~0ull, 0ull);
        if constexpr (ROW4) {        // a byte a warp: 8 rows
          rows = make_ulonglong2(mk[0], mk[2]);
        } else {
          const unsigned long long m0 = mk[0], m1 = mk[1], d0 = mk[2], d1 = mk[3];
          if (__any_sync(0xffffffffu, (m0 & m1) != 0x0f0f0f0f0f0f0f0full || (d0 | d1) != 0))
            rows = make_ulonglong2(halves(m0, m1), halves(d0, d1));
        }
        // the value product before the last is done with its weights, in whose place this block's will be
        if (n >= 2) ok = warp_wait(bar(EMPTY + Place::of(2 * n - 3).at), Place::of(2 * n - 3).phase, stop, a.status);
        if (ok) ok = warp_wait(bar(SFULL + (n & 1)), (n >> 1) & 1, stop, a.status);
        if (!ok) break;
        // also of a warp without rows: the tile's last scores are worked out before the next Q takes its place
        tc_fence_after();
        if (idle) {
          if (lane == 0) {
            mbar_arrive(bar(SEMPTY + (n & 1)));
            mbar_arrive(bar(PFULL + (n & 1)));
          }
          continue;
        }
        float v[16];
        tmem_ld_16x32(tS + 64 * (n & 1), v);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(SEMPTY + (n & 1)));
        uint32_t p[8];
        float alpha[2];
        st.weights(v, (blk - i) * kChunkBlk, rows, most + (n & 1) * 128, p, alpha);
        // O may be rescaled once the value product before this one is done
        if (i > 0 && __any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
          ok = warp_wait(bar(EMPTY + Place::of(2 * n - 1).at), Place::of(2 * n - 1).phase, stop, a.status);
          if (!ok) {
            held = 1;
            break;
          }
          tc_fence_after();
          rescale_half(tO, alpha[0], alpha[1], half);
        }
        tmem_st_16x16(tP + 32 * (n & 1), p);
        tmem_st_16x16(tP + 32 * (n & 1) + kUpper, p);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(PFULL + (n & 1)));
      }
      if (!ok) break;
      // all scores of the tile have been seen: the next one's Q may take this one's place
      if (end < x1) give_q(t + 1);
      ok = warp_wait(bar(EMPTY + Place::of(2 * n - 1).at), Place::of(2 * n - 1).phase, stop, a.status);
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
        const int end = min(x1, line.cum(t + 1));
        if (16 * quarter < line.tile(t).z)
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

template <bool MODS, bool ROW4>
cudaError_t launch(const ChunkArgs& a, const ChunkPlan& p, int workers, cudaStream_t stream) {
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    if (!done[dev]) {
      e = cudaFuncSetAttribute(single_kernel<MODS, ROW4>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (e != cudaSuccess) return e;
      // the register split assumes the launch's share: a build that differs is refused,
      // since its increase would never be granted
      cudaFuncAttributes fa;
      e = cudaFuncGetAttributes(&fa, single_kernel<MODS, ROW4>);
      if (e != cudaSuccess) return e;
      if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidKernelImage;
      done[dev] = true;
    }
  }
  return launch_programmatic(single_kernel<MODS, ROW4>, dim3(workers), dim3(kThreads), kSmem, stream, a, p);
}

}  // namespace

cudaError_t launch_chunk_single(const ChunkArgs& a, const ChunkPlan& p, int workers, cudaStream_t stream) {
  const bool mods = a.cap > 0.f || a.slopes != nullptr;
  if (is_row4(a.stride)) return mods ? launch<true, true>(a, p, workers, stream) : launch<false, true>(a, p, workers, stream);
  return mods ? launch<true, false>(a, p, workers, stream) : launch<false, false>(a, p, workers, stream);
}

}  // namespace smla
