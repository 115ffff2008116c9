// Attention of a chunk of new tokens over the paged cache (smla_chunk_attention).
// Declared and documented in include/smla.h.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/smla.h"
#include "smla_cache_rows.cuh"
#include "smla_chunk.h"
#include "smla_internal.h"
#include "smla_ptx.cuh"

namespace smla {
namespace {

// ---------------------------------------------------------------------------
// Plan: one CTA, 6 to 7 us cold (a launch, three dependent loads, block-wide sums), within the
// expansion's launch where there is one.  Equal shares of the block line, whatever the lengths
// and masks: no SM waits for the longest sequence.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
// kMinShare, the least blocks of a share, pays for its query tile and its partial result: 4 x 4 tokens of
// 1,001: 33.0, 29.3, 31.6 and 35.9 us with 1, 2, 4 and 8.
// A border within kSnap blocks of a tile's end moves there (by a quarter of a share at
// most): a piece of a tile costs its 256 rows of Q and 458 KB of partial results, which leave an SM
// at 28 bytes a cycle, as much as four blocks.  Seven ragged sequences of 16 heads: 68.0, 65.3,
// 59.5, 59.4 and 59.5 us with 0, 1, 2, 3 and 6; three of 700 tokens in a window 156, 153, 151,
// 147 and 146; single tokens do not mind.

// Exclusive sum over the CTA; *total gets the sum.
__device__ long long block_sum(long long v, long long* total, long long* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  if (warp == 0) {
    long long w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  *total = warp_sums[31];
  return s - v + (warp > 0 ? warp_sums[warp - 1] : 0);
}

constexpr int kPlanSeqs = 1024;    // sequences and tiles whose plan fits in shared memory
constexpr int kPlanTiles = 2048;
struct PlanShared {
  long long sums[32];
  int32_t tile[kPlanSeqs + 1], first[kPlanSeqs], last[kPlanSeqs], len[kPlanSeqs];
  int32_t cum[kPlanTiles + 1];
};

// By one CTA of kPlanThreads.  tile_rows: (token, head) rows of a tile; workers: shares of
// the line.  Latency is all that counts here (a few dependent loads and block-wide sums), so
// what the tiles need of their sequences, and the line, stay in shared memory in usual calls.
__device__ void make_plan(const ChunkArgs& a, const ChunkPlan& p, int tile_rows, int workers,
                          PlanShared& sh) {
  const bool few = a.B <= kPlanSeqs;
  long long tiles = 0, blocks = 0;
  bool wrong = false;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    const Sequence s = sequence(a, b);
    wrong |= s.wrong;
    const int nt = (s.n * a.H + tile_rows - 1) / tile_rows;      // total_q * H < 2^30
    long long t_all, b_all;
    const long long t0 = tiles + block_sum(nt, &t_all, sh.sums);
    const long long s0 = blocks + block_sum(s.blocks, &b_all, sh.sums);
    if (b < a.B) {
      const int len = seq_len(p, s, s0);
      if (len != s.len) atomicCAS(a.status, 0, SMLA_ERR_INDEX_RANGE);
      p.tile_base[b] = static_cast<int>(t0);
      p.seq_base[b] = seq_base(p, s0);
      p.seq_len[b] = len;
      if (few) {
        sh.tile[b] = static_cast<int>(t0);
        sh.first[b] = s.first;
        sh.last[b] = s.first + s.n;
        sh.len[b] = len;
      }
    }
    tiles += t_all;
    blocks += b_all;
  }
  if (threadIdx.x == 0) {
    p.tile_base[a.B] = static_cast<int>(tiles);
    p.seq_base[a.B] = seq_base(p, blocks);
    if (few) sh.tile[a.B] = static_cast<int>(tiles);
  }
  // Offsets in order and within q give each entry to one sequence at most, and no more tiles than
  // the workspace has room for; with others the call does nothing.
  if (__syncthreads_or(wrong)) {
    tiles = 0;
    if (threadIdx.x == 0) atomicCAS(a.status, 0, SMLA_ERR_INDEX_RANGE);
  }
  const bool short_line = tiles <= kPlanTiles;
  long long line = 0;
  for (int t0 = 0; t0 < static_cast<int>(tiles); t0 += kPlanThreads) {
    const int t = t0 + static_cast<int>(threadIdx.x);
    int4 tile = make_int4(0, 0, 0, 0);
    int n = 0;
    if (t < tiles) {
      int b, first, last, len, base;
      if (few) {
        b = find_last_le(sh.tile, a.B + 1, t);
        first = sh.first[b];
        last = sh.last[b];
        len = sh.len[b];
        base = sh.tile[b];
      } else {
        b = find_last_le(p.tile_base, a.B + 1, t);
        const Sequence s = sequence(a, b);
        first = s.first;
        last = s.first + s.n;
        len = p.seq_len[b];
        base = p.tile_base[b];
      }
      const int row = first * a.H + (t - base) * tile_rows;
      const int rows = min(tile_rows, last * a.H - row);
      int blk;
      tile_blocks(a, b, row, rows, len, &blk, &n);
      tile = make_int4(b, row, rows, blk);
    }
    long long all;
    const long long at = line + block_sum(n, &all, sh.sums);
    if (t < tiles) {
      const int cum = static_cast<int>(min(at, 0x7fffffffll));
      p.tile[t] = tile;
      p.cum[t] = cum;
      if (short_line) sh.cum[t] = cum;
    }
    line += all;
  }
  if (line > (1 << 30)) {     // far past any call that ends within hours: positions on the line stay ints
    line = 0;
    tiles = 0;
    if (threadIdx.x == 0) atomicCAS(a.status, 0, SMLA_ERR_UNSUPPORTED_SHAPE);
  }
  const int per = max(kMinShare, static_cast<int>((line + workers - 1) / workers));
  if (threadIdx.x == 0) {
    p.cum[tiles] = static_cast<int>(line);
    if (short_line) sh.cum[tiles] = static_cast<int>(line);
  }
  __syncthreads();
  // where each share begins, and the tile there, so that nobody else has to search
  const int32_t* cum = short_line ? sh.cum : p.cum;
  const int c = static_cast<int>(threadIdx.x), snap = min(kSnap, per / 4);
  int32_t* border = sh.first;
  int t = -1;
  if (c <= workers) {
    int x = static_cast<int>(min(static_cast<long long>(c) * per, line));
    if (x < line) {
      t = find_last_le(cum, static_cast<int>(tiles) + 1, x);
      if (x - cum[t] <= snap) x = cum[t];
      else if (cum[t + 1] - x <= snap) x = cum[++t];
      if (x == line) t = -1;
    }
    border[c] = x;
    p.begin[c] = x;
    if (c < workers) p.start[c] = t;
  }
  __syncthreads();
  // the cut tiles, found at the first share that begins inside each
  bool cut = false;
  int4 piece = make_int4(0, 0, 0, 0);
  if (c > 0 && c < workers && t >= 0) {
    cut = cum[t] < border[c] && border[c - 1] <= cum[t];
    if (cut) {
      const int4 tile = p.tile[t];
      piece = make_int4(tile.y, tile.z, c - 1, find_last_le(border, workers + 1, cum[t + 1] - 1));
    }
  }
  long long cuts;
  const long long k = block_sum(cut ? 1 : 0, &cuts, sh.sums);
  if (cut) p.cut[k] = piece;
  if (threadIdx.x == 0) {
    p.head[0] = static_cast<int>(tiles);
    p.head[1] = static_cast<int>(line);
    p.head[2] = static_cast<int>(cuts);
  }
}

__global__ void __launch_bounds__(kPlanThreads, 1)
    plan_kernel(const ChunkArgs a, const ChunkPlan p, int tile_rows, int workers) {
  __shared__ PlanShared sh;
  grid_dep_wait();
  grid_dep_launch();
  make_plan(a, p, tile_rows, workers, sh);
}

// ---------------------------------------------------------------------------
// Expanded copy: the rows of each sequence in the order of its positions, bf16.  The e4m3
// values times their powers of two are exact in bf16.  A CTA takes a block of 64 rows, a warp
// two of them; lane l < 28 holds columns 16 l .. 16 l + 15, lanes 28..31 the rope.  Bound by
// the launch and one trip to memory: 7.5 us for 8,192 rows (1.6 KB each), 11 us for 21,007.
// ---------------------------------------------------------------------------
__device__ __forceinline__ bool not_finite(uint32_t bf16x2) {
  return (bf16x2 & 0x7f80u) == 0x7f80u || (bf16x2 & 0x7f800000u) == 0x7f800000u;
}

// CTA 0 makes the plan meanwhile; the others find the sequences' places by themselves (the
// same sums over the batch), so that one launch does both.
constexpr int kExpandRows = 2;     // rows of a block that a warp expands at once: 32 warps, 64 rows
template <bool ROW4>
__global__ void __launch_bounds__(kPlanThreads, 1)
    expand_kernel(const ChunkArgs a, const ChunkPlan p, int tile_rows, int workers) {
  __shared__ PlanShared sh;
  __shared__ uint32_t mapped[32], odd[32];
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x == 0) {
    make_plan(a, p, tile_rows, workers, sh);
    return;
  }
  // sh.first: first block of each sequence, sh.last: its visible positions; in rounds of
  // kPlanSeqs sequences
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long blocks = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanSeqs) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    const Sequence s = sequence(a, b);
    long long all;
    const long long s0 = blocks + block_sum(s.blocks, &all, sh.sums);
    sh.first[threadIdx.x] = seq_base(p, s0);
    sh.last[threadIdx.x] = seq_len(p, s, s0);
    const int begin = seq_base(p, blocks), end = seq_base(p, blocks + all);
    blocks += all;
    __syncthreads();
    const int seqs = min(kPlanSeqs, a.B - b0);
    // blocks [begin, end) in turn; with the last round also the one behind the copy: zeros,
    // for the sequences that found no room
    const int stop = b0 + kPlanSeqs >= a.B ? end + 1 : end;
    const int step = gridDim.x - 1;
    int g = begin + (static_cast<int>(blockIdx.x) - 1 - begin % step + step) % step;
    for (; g < stop; g += step) {
      const bool real = g < end;
      const int64_t out_blk = real ? g : p.cap_blocks;
      int i = 0, s0 = 0, len = 0;
      if (real) {
        // the last sequence that begins at or before g and has blocks
        i = find_last_le(sh.first, seqs, g);
        s0 = (g - sh.first[i]) * kChunkBlk;
        len = sh.last[i];
      }
      // lane j < kExpandRows: the pool row of position s0 + kExpandRows warp + j
      long long row = -1;
      const int pos = s0 + kExpandRows * warp + lane;
      if (lane < kExpandRows && pos < len) {
        const int page = pos / a.page_size;
        if (page >= a.max_pages) {
          atomicCAS(a.status, 0, SMLA_ERR_INDEX_RANGE);
        } else {
          const int phys = __ldg(a.table + static_cast<int64_t>(b0 + i) * a.max_pages + page);
          if (phys >= 0) {
            row = static_cast<long long>(phys) * a.page_size + (pos - page * a.page_size);
            if (row >= a.num_rows) {
              row = -1;
              atomicCAS(a.status, 0, SMLA_ERR_INDEX_RANGE);
            }
          }
        }
      }
      const uint32_t have = __ballot_sync(0xffffffffu, row >= 0);
      uint32_t poison = 0;
      RowLane in[kExpandRows];
#pragma unroll
      for (int j = 0; j < kExpandRows; ++j) {
        const long long r = __shfl_sync(0xffffffffu, row, j);
        load_row<ROW4>(r >= 0 ? a.pool + r * a.stride : nullptr, in[j]);
      }
#pragma unroll
      for (int j = 0; j < kExpandRows; ++j) {
        uint32_t o[8];
        row_values<ROW4>(in[j], o);
        bool bad = false;      // a NaN (a scale byte of 255 makes NaN), or past bf16's largest value
#pragma unroll
        for (int k = 0; k < 8; ++k) bad |= not_finite(o[k]);
        if (__any_sync(0xffffffffu, bad)) {
          poison |= 1u << j;
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] = 0;
        }
        uint4* dst = reinterpret_cast<uint4*>(p.kv + (out_blk * kChunkBlk + kExpandRows * warp + j) * kQkDim + 16 * lane);
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
      }
      if (lane == 0) {
        mapped[warp] = have & ((1u << kExpandRows) - 1u);
        odd[warp] = poison;
      }
      __syncthreads();
      if (warp == 0) {
        // warp w's bits at kExpandRows w: the lower 16 warps make the low words
        const uint32_t m = mapped[lane] << (kExpandRows * (lane & 15)), q = odd[lane] << (kExpandRows * (lane & 15));
        const uint32_t m0 = __reduce_or_sync(0xffffffffu, lane < 16 ? m : 0u), m1 = __reduce_or_sync(0xffffffffu, lane < 16 ? 0u : m);
        const uint32_t q0 = __reduce_or_sync(0xffffffffu, lane < 16 ? q : 0u), q1 = __reduce_or_sync(0xffffffffu, lane < 16 ? 0u : q);
        if (lane == 0)
          p.seen[out_blk] = make_ulonglong2(m0 | static_cast<unsigned long long>(m1) << 32,
                                            q0 | static_cast<unsigned long long>(q1) << 32);
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------------------
// Merge: the partial results of the tiles that a share's border cuts.  Grid (row groups, cut
// tiles).  A row is joined by ROW_WARPS warps, each taking every
// ROW_WARPS-th partial result: a long context over one tile of few rows has as many partial
// results as there are workers, and one warp reading them in turn would be all latency.
// Bound by latency and L2 (the parts were written just before): 16 us for the 75 tiles of 256
// rows that 76 pairs cut (69 MB), 8 us behind single tokens.  Rows of few tiles: 8 warps each
// (15 us with 2 for two tiles of 76 parts, 8 with 8); else one warp each, as the parts are two
// or three.
// ---------------------------------------------------------------------------
struct Part {             // a lane's share of a partial result: float4 lane + 28 k of 112
  float4 v[4];
};
__device__ __forceinline__ void add_scaled(Part& x, float w, const Part& y) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x.v[k].x = fmaf(w, y.v[k].x, x.v[k].x);
    x.v[k].y = fmaf(w, y.v[k].y, x.v[k].y);
    x.v[k].z = fmaf(w, y.v[k].z, x.v[k].z);
    x.v[k].w = fmaf(w, y.v[k].w, x.v[k].w);
  }
}
template <int ROW_WARPS>
__global__ void __launch_bounds__(256) merge_kernel(const ChunkArgs a, const ChunkPlan p, int tile_rows) {
  constexpr int kRows = 8 / ROW_WARPS;          // rows of a CTA
  constexpr int kLanes = 28;                    // of 16 bytes: 4 x 28 are a row
  __shared__ float4 part[ROW_WARPS > 1 ? 8 : 1][4][kLanes];     // each warp's sum over its partial results
  __shared__ float weight[8];
  grid_dep_wait();
  grid_dep_launch();
  int4 cut;                               // first row of the tile, rows, first and last worker
  if (is_even<true>(p)) {
    // tile y, or, of more tiles than borders, the one that border y + 1 is the first inside
    const int n = p.even.blocks, y = blockIdx.y;
    const bool by_tile = a.B * p.even.tiles < kMaxSms;
    const int t = by_tile ? y : plan_begin<true>(p, y + 1) / n, from = t * n;
    if (!by_tile) {
      const int border = plan_begin<true>(p, y + 1);
      if (border >= p.even.line || border == from || plan_begin<true>(p, y) > from) return;
    }
    auto share = [&](int x) {        // the last that begins at block x or before: a border moves by less than a share
      int c = p.even.pieces > 0 ? x / n * p.even.pieces : x / p.even.per;
      while (c > 0 && plan_begin<true>(p, c) > x) --c;
      while (c + 1 < kMaxSms && plan_begin<true>(p, c + 1) <= x) ++c;
      return c;
    };
    const int first = by_tile ? share(from) : y, last = p.even.pieces > 0 ? first + p.even.pieces - 1 : share(from + n - 1);
    if (first == last) return;
    const int4 tile = plan_tile<true>(p, t);
    cut = make_int4(tile.y, tile.z, first, last);
  } else {
    const int cuts = p.head[2];
    cut = p.cut[blockIdx.y];
    if (static_cast<int>(blockIdx.y) >= cuts) return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * kRows + warp / ROW_WARPS;
  if (static_cast<int>(blockIdx.x) * kRows >= cut.y) return;
  const int first = cut.z, last = cut.w;
  // slot of worker c: its share begins inside the tile (0), or the tile inside its share (1)
  auto at = [&](int c) { return static_cast<int64_t>(2 * c + (c == first ? 1 : 0)) * tile_rows + row; };
  const bool live = row < cut.y;
  auto load = [&](int c, Part& x) {
    const float4* o = reinterpret_cast<const float4*>(p.o_part + at(c) * kNope) + lane;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      x.v[k] = live && lane < kLanes && c <= last ? __ldcg(o + kLanes * k) : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  // two partial results are on their way while the weights are worked out
  const int c0 = first + warp % ROW_WARPS;
  Part x0, x1, acc = {};
  load(c0, x0);
  load(c0 + ROW_WARPS, x1);
  const float mine = live && first + lane <= last ? p.lse_part[at(first + lane)] : -INFINITY;
  float top = mine;
  if (live)
    for (int c = first + 32 + lane; c <= last; c += 32) top = fmaxf(top, p.lse_part[at(c)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float shift = top == -INFINITY ? 0.f : top;
  float sum = 0.f;
  for (int c = c0; c <= last; c += 2 * ROW_WARPS) {
    const int c1 = c + ROW_WARPS;
    const float z0 = __shfl_sync(0xffffffffu, mine, (c - first) & 31), z1 = __shfl_sync(0xffffffffu, mine, (c1 - first) & 31);
    const float w0 = live ? expf((c - first < 32 ? z0 : p.lse_part[at(c)]) - shift) : 0.f;
    const float w1 = live && c1 <= last ? expf((c1 - first < 32 ? z1 : p.lse_part[at(c1)]) - shift) : 0.f;
    add_scaled(acc, w0, x0);
    add_scaled(acc, w1, x1);
    sum += w0;
    sum += w1;
    load(c + 2 * ROW_WARPS, x0);
    load(c1 + 2 * ROW_WARPS, x1);
  }
  if constexpr (ROW_WARPS > 1) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (lane < kLanes) part[warp][k][lane] = acc.v[k];
    if (lane == 0) weight[warp] = sum;
    __syncthreads();
    if (warp % ROW_WARPS != 0) return;
#pragma unroll
    for (int w = 1; w < ROW_WARPS; ++w) {       // in a fixed order: the same bits every time
      sum += weight[warp + w];
      Part x;
#pragma unroll
      for (int k = 0; k < 4; ++k) x.v[k] = part[warp + w][k][min(lane, kLanes - 1)];
      add_scaled(acc, 1.f, x);
    }
  }
  if (!live) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t orow = static_cast<int64_t>(cut.x) + row;
  uint2* out = reinterpret_cast<uint2*>(a.out + orow * kNope) + lane;
  if (lane < kLanes) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      out[kLanes * k] = make_uint2(pack_bf16(acc.v[k].x * inv, acc.v[k].y * inv), pack_bf16(acc.v[k].z * inv, acc.v[k].w * inv));
  }
  if (lane == 0) a.lse[orow] = sum == 0.f ? -INFINITY : shift + logf(sum);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_chunk(const smla_chunk_params* p) {
  if (p == nullptr || p->reserved != 0) return SMLA_ERR_INVALID_ARG;
  if (p->batch < 1 || p->total_q < 1 || p->page_size < 1 || p->max_pages < 1 || p->num_rows < 1 ||
      p->max_kv_tokens < 1)
    return SMLA_ERR_INVALID_ARG;
  if (!row_stride_ok(p->kv_row_stride)) return SMLA_ERR_INVALID_ARG;
  if (!(std::isfinite(p->softmax_scale) && p->softmax_scale > 0.f)) return SMLA_ERR_INVALID_ARG;
  if (!(std::isfinite(p->logit_cap) && p->logit_cap >= 0.f)) return SMLA_ERR_INVALID_ARG;
  if (p->num_heads != 16 && p->num_heads != 32 && p->num_heads != 64 && p->num_heads != 128)
    return SMLA_ERR_UNSUPPORTED_SHAPE;
  if (p->batch > 65535 || p->max_kv_tokens > (int64_t{1} << 30) || p->num_rows > (int64_t{1} << 31) ||
      p->kv_row_stride >= (int64_t{1} << 31) || static_cast<int64_t>(p->total_q) * p->num_heads >= (int64_t{1} << 30))
    return SMLA_ERR_UNSUPPORTED_SHAPE;
  return SMLA_OK;
}

constexpr int kMaxPairs = kMaxSms / 2;
size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Which kernel: pairs once a sequence brings a full tile of 256 rows on average.  Single against
// pairs, 16 sequences of 16,000 and 64 heads: 1 token 90 and 184 us, 2 tokens 126 and 161, 4
// tokens 214 and 160; 16 tokens of 16 heads over 8,000 93 and 88; 1 token of 128 heads 60 and 70.
// Over 4-bit rows, which cost the single kernel less, from more than a full tile: of 64 heads, 4 x 4 tokens of 1,001
// 24.7 and 26.8, 16 x 4 of 16,000 183 and 199, 32 x 4 of 500 39.1 and 34.8; 4 x 5 of 1,001 30.8 and 28.7, 3 x 5 of
// 19,717 70 and 81, 8 x 8 of 4,000 67 and 60; 16 x 16 of 16 heads and 8,000 106 and 116.
// The length decides too, which the rule does not look at: 3 x 5 of 19,717 and 32 x 4 of 500 are on their slower side.
// All of batches whose sequences bring the same number of tokens; mixed ones are not measured.
bool use_pairs(const smla_chunk_params* p) {
  const int64_t rows = static_cast<int64_t>(p->total_q) * p->num_heads, full = static_cast<int64_t>(kPairRows) * p->batch;
  return is_row4(p->kv_row_stride) ? rows > full : rows >= full;
}

// The workspace of a call; base may be null to size it.
size_t lay_out(const smla_chunk_params* p, char* base, ChunkPlan* plan) {
  size_t at = 0;
  plan->even = {};
  // the tiles of sequences that all end inside one: no less than there are
  plan->few = !use_pairs(p) && p->batch <= kFewTiles &&
              (static_cast<int64_t>(p->total_q) * p->num_heads +
               static_cast<int64_t>(p->batch) * (p->num_heads < kSingleRows ? kSingleRows - p->num_heads : 0)) /
                      kSingleRows <= kFewTiles;
  auto take = [&](size_t bytes) {
    char* q = base + at;
    at += round256(bytes);
    return q;
  };
  const size_t B = p->batch;
  const size_t tiles = (static_cast<size_t>(p->total_q) * p->num_heads + kSingleRows - 1) / kSingleRows + B;
  const int64_t cap = (p->max_kv_tokens + kChunkBlk - 1) / kChunkBlk + p->batch;
  plan->cap_blocks = cap;
  plan->head = reinterpret_cast<int32_t*>(take(256));
  plan->tile = reinterpret_cast<int4*>(take(16 * tiles));
  plan->cum = reinterpret_cast<int32_t*>(take(4 * (tiles + 1)));
  plan->tile_base = reinterpret_cast<int32_t*>(take(4 * (B + 1)));
  plan->seq_base = reinterpret_cast<int32_t*>(take(4 * (B + 1)));
  plan->seq_len = reinterpret_cast<int32_t*>(take(4 * B));
  plan->start = reinterpret_cast<int32_t*>(take(4 * kMaxSms));
  plan->begin = reinterpret_cast<int32_t*>(take(4 * (kMaxSms + 1)));
  plan->cut = reinterpret_cast<int4*>(take(16 * kMaxSms));
  const size_t parts = use_pairs(p) ? 2 * kMaxPairs * kPairRows : 2 * kMaxSms * kSingleRows;
  plan->lse_part = reinterpret_cast<float*>(take(4 * parts));
  plan->o_part = reinterpret_cast<float*>(take(4 * parts * kNope));
  // the expanded copy, which only pairs read
  const size_t copies = use_pairs(p) ? static_cast<size_t>(cap + 1) : 0;
  plan->seen = reinterpret_cast<ulonglong2*>(take(16 * copies));
  plan->kv = reinterpret_cast<uint16_t*>(take(copies * kChunkBlk * kQkDim * 2));
  return at;
}

cudaError_t launch_merge(const ChunkArgs& a, const ChunkPlan& p, int rows, int workers, cudaStream_t s) {
  if (workers < 2) return cudaSuccess;
  // few tiles: many partial results a row (see the kernel)
  const int64_t tiles = (static_cast<int64_t>(a.T) * a.H + rows - 1) / rows + a.B;
  const int64_t even = static_cast<int64_t>(a.B) * p.even.tiles, most = p.even.blocks > 0 ? even : tiles;
  const unsigned cuts = static_cast<unsigned>(most < workers - 1 ? most : workers - 1);
  if (tiles * 4 <= workers)
    return launch_programmatic(merge_kernel<8>, dim3(rows, cuts), dim3(256), 0, s, a, p, rows);
  return launch_programmatic(merge_kernel<1>, dim3(rows / 8, cuts), dim3(256), 0, s, a, p, rows);
}

cudaError_t launch_pair_path(const ChunkArgs& a, const ChunkPlan& p, cudaStream_t s) {
  int workers = 0;
  cudaError_t e = pair_workers(&workers);
  if (e != cudaSuccess) return e;
  if (workers > kMaxPairs) workers = kMaxPairs;
  const int64_t blocks = p.cap_blocks + 1;
  const unsigned grid = 1 + static_cast<unsigned>(blocks < kMaxSms - 1 ? blocks : kMaxSms - 1);
  e = launch_programmatic(is_row4(a.stride) ? expand_kernel<true> : expand_kernel<false>, dim3(grid), dim3(kPlanThreads), 0,
                          s, a, p, kPairRows, workers);
  if (e != cudaSuccess) return e;
  e = launch_chunk_pair(a, p, workers, s);
  return e == cudaSuccess ? launch_merge(a, p, kPairRows, workers, s) : e;
}

cudaError_t launch_single_path(const ChunkArgs& a, const ChunkPlan& p, cudaStream_t s) {
  const int workers = kMaxSms;
  cudaError_t e = cudaSuccess;
  if (p.even.blocks == 0 && !p.few)
    e = launch_programmatic(plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a, p, kSingleRows, workers);
  if (e == cudaSuccess) e = launch_chunk_single(a, p, workers, s);
  return e == cudaSuccess ? launch_merge(a, p, kSingleRows, workers, s) : e;
}

// Sparse decode over 4-bit rows as a chunk of one token a sequence that sees topk listed rows.
smla_chunk_params sparse_as_chunk(const smla_params* p) {
  return {p->batch, p->num_heads, p->batch, 1, p->topk, 0, p->num_rows, p->kv_row_stride,
          static_cast<int64_t>(p->batch) * (((p->topk - 1) / kChunkBlk + 1) * kChunkBlk), p->softmax_scale, 0.f};
}

}  // namespace

size_t sparse4_workspace(const smla_params* p) {
  const smla_chunk_params c = sparse_as_chunk(p);
  ChunkPlan plan;
  return lay_out(&c, nullptr, &plan);
}

int launch_sparse4(const void* q, const void* kv, const int32_t* indices, const int32_t* block_table, int max_pages,
                   int page_size, void* out, float* lse, const smla_params* p, void* workspace, cudaStream_t stream) {
  int* status = nullptr;
  if (status_word_address(&status) != cudaSuccess) return SMLA_ERR_CUDA;
  const smla_chunk_params c = sparse_as_chunk(p);
  const ChunkArgs a = {static_cast<const uint16_t*>(q), static_cast<const uint8_t*>(kv), indices, nullptr, nullptr,
                       nullptr, nullptr, nullptr, static_cast<__nv_bfloat16*>(out), lse, c.batch, c.num_heads,
                       c.total_q, 1, c.max_pages, c.num_rows, c.kv_row_stride, c.softmax_scale, 0.f, status,
                       fault_block(), p->topk, block_table, max_pages, page_size};
  ChunkPlan plan;
  lay_out(&c, static_cast<char*>(workspace), &plan);
  const int blocks = (p->topk - 1) / kChunkBlk + 1, tiles = (p->num_heads - 1) / kSingleRows + 1;
  const int line = p->batch * tiles * blocks, share = (line + kMaxSms - 1) / kMaxSms;      // 65,535 * 2 * 1,024 at most
  const int per = share > kMinShare ? share : kMinShare;
  // Shares that end with their tiles, some SMs left over, or shares along the line, whose change of tile costs as
  // much as kTileChange blocks (13,000 cycles: Q, and results that the next tile's scores wait for).  32 queries
  // of 2,048 and 64 heads: 4 shares of 8 blocks each (taken: 29.6 us, 32.7 along the line), or 147 of 7; 96 of 999 and 16
  // heads: one of 16, or 140 of 11 (taken: 16 is more than 11 + 4; the other is not measured).
  constexpr int kTileChange = 4;
  int pieces = p->batch * tiles <= kMaxSms ? kMaxSms / (p->batch * tiles) : 0;
  if (pieces > (blocks + 1) / kMinShare) pieces = (blocks + 1) / kMinShare;
  if (pieces > 0 && (blocks - 1) / pieces + 1 > per + kTileChange) pieces = 0;
  plan.even = {blocks, tiles, p->num_heads, pieces, per, line, per / 4 < kSnap ? per / 4 : kSnap};
  return launch_single_path(a, plan, stream) == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

}  // namespace smla

using namespace smla;   // NOLINT: the entry points below are this file's own

extern "C" {

int smla_chunk_workspace_size(const smla_chunk_params* p, size_t* bytes) {
  const int st = check_chunk(p);
  if (st != SMLA_OK) return st;
  if (bytes == nullptr) return SMLA_ERR_INVALID_ARG;
  ChunkPlan plan;
  *bytes = lay_out(p, nullptr, &plan);
  return SMLA_OK;
}

int smla_chunk_attention(const void* q, const void* kv_pages, const int32_t* block_table,
                         const int32_t* cu_q, const int32_t* kv_lens, const int32_t* vis_begin,
                         const int32_t* vis_end, const float* slopes, void* out, float* lse,
                         const smla_chunk_params* p, void* workspace, size_t workspace_bytes,
                         smla_stream_t stream) {
  int st = check_chunk(p);
  if (st != SMLA_OK) return st;
  if (q == nullptr || kv_pages == nullptr || block_table == nullptr || cu_q == nullptr ||
      kv_lens == nullptr || out == nullptr || lse == nullptr || workspace == nullptr)
    return SMLA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv_pages, 16) || !aligned(out, 16) || !aligned(workspace, 256) ||
      !aligned(block_table, 4) || !aligned(cu_q, 4) || !aligned(kv_lens, 4) || !aligned(vis_begin, 4) ||
      !aligned(vis_end, 4) || !aligned(slopes, 4) || !aligned(lse, 4))
    return SMLA_ERR_INVALID_ARG;
  size_t need = 0;
  st = smla_chunk_workspace_size(p, &need);
  if (st != SMLA_OK) return st;
  if (workspace_bytes < need) return SMLA_ERR_WORKSPACE_TOO_SMALL;
  st = check_device();
  if (st != SMLA_OK) return st;
  int* status = nullptr;
  if (status_word_address(&status) != cudaSuccess) return SMLA_ERR_CUDA;
  const ChunkArgs a = {static_cast<const uint16_t*>(q), static_cast<const uint8_t*>(kv_pages),
                       block_table, cu_q, kv_lens, vis_begin, vis_end, slopes,
                       static_cast<__nv_bfloat16*>(out), lse, p->batch, p->num_heads, p->total_q,
                       p->page_size, p->max_pages, p->num_rows, p->kv_row_stride, p->softmax_scale,
                       p->logit_cap, status, fault_block(), 0, nullptr, 0, 0};
  ChunkPlan plan;
  lay_out(p, static_cast<char*>(workspace), &plan);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = use_pairs(p) ? launch_pair_path(a, plan, s) : launch_single_path(a, plan, s);
  return e == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

}  // extern "C"
