// What the translation units of the chunk attention share: the arguments of a call, its
// plan in the workspace, and the launches.  Not part of the public ABI.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/smla.h"
#include "smla_internal.h"
#include "smla_ptx.cuh"

namespace smla {

constexpr int kChunkBlk = 64;     // positions of a block
constexpr int kMaxSms = 152;      // SMs of the GPU that this library is for: the workers that a workspace has room for

struct ChunkArgs {
  const uint16_t* q;
  const uint8_t* pool;
  const int32_t *table, *cu_q, *kv_lens, *vis_begin, *vis_end;
  const float* slopes;
  __nv_bfloat16* out;
  float* lse;
  int B, H, T, page_size, max_pages;
  int64_t num_rows, stride;
  float scale, cap;
  int* status;
  int fault_block;       // test hook: the block of each share that one warp does not report (-1: none)
  // Sparse decode: every sequence is one token that sees `listed` slots; `table` lists their rows (pages
  // of one row), or, with `pages`, their positions in the sequence.  cu_q and kv_lens are not read.
  int listed;            // 0: not sparse
  const int32_t* pages;  // [B, max_listed_pages] or null
  int max_listed_pages, listed_page_size;
};

// The plan of a call: the (token, head) rows of each sequence cut into tiles, each tile's
// visible blocks of 64 positions laid end to end over all tiles, and that line cut into
// equal shares, one a worker.  A tile that lies in one share is finished by its worker;
// the others leave partial results that the merge joins.
struct ChunkPlan {
  int32_t* head;         // [0] tiles, [1] blocks on the line, [2] cut tiles
  int4* tile;            // sequence, first row (token * H + head), rows, first block
  int32_t* cum;          // [tiles + 1] start of each tile on the line
  int32_t* start;        // [workers] the tile at the start of each share, -1 behind the line
  int32_t* begin;        // [workers + 1] where each share starts on the line
  int4* cut;             // [cut tiles] first row, rows, first and last worker
  int32_t* tile_base;    // [B + 1] first tile of each sequence
  int32_t* seq_base;     // [B + 1] first block of each sequence in the expanded copy
  int32_t* seq_len;      // [B] positions of each sequence that can be seen
  float* o_part;         // [2 workers][rows of a tile][448]
  float* lse_part;       // [2 workers][rows of a tile]
  ulonglong2* seen;      // [blocks] of each expanded block: the mapped positions, and those
                         // of them whose row has a value that is not finite
  uint16_t* kv;          // [blocks][64][512] bf16: the expanded copy
  int64_t cap_blocks;    // blocks of the expanded copy, not counting one of zeros behind
  // Single kernel: 32 sequences and tiles at most, so that a warp of each CTA works the plan out for itself, into
  // shared memory, and the first one what the merge needs
  bool few;
  // Sparse decode: every tile has as many blocks, so that the plan follows from its number (blocks 0: it
  // lies in memory, above).
  struct Even {
    int blocks, tiles, heads;      // of a tile; of a sequence
    int pieces;                    // shares of a tile, if whole shares make up each; else 0, and
    int per, line, snap;           // shares along the line as make_plan has them
  } even;
};

// Blocks of a share, and how far a border moves to a tile's end (see make_plan).
constexpr int kMinShare = 2, kSnap = 3;

// The plan's parts, of sparse decode where EVEN allows for it.
template <bool EVEN>
__device__ __forceinline__ bool is_even(const ChunkPlan& p) {
  return EVEN && p.even.blocks > 0;
}
template <bool EVEN>
__device__ __forceinline__ int plan_begin(const ChunkPlan& p, int worker) {
  if (!is_even<EVEN>(p)) return p.begin[worker];
  if (p.even.pieces > 0) {
    const int t = worker / p.even.pieces;
    return min(p.even.line, t * p.even.blocks + (worker - t * p.even.pieces) * p.even.blocks / p.even.pieces);
  }
  const int n = p.even.blocks, x = min(worker * p.even.per, p.even.line), rest = x % n;
  return rest <= p.even.snap ? x - rest : n - rest <= p.even.snap ? x + n - rest : x;
}
template <bool EVEN>
__device__ __forceinline__ int plan_start(const ChunkPlan& p, int worker, int begin) {
  return is_even<EVEN>(p) ? begin / p.even.blocks : p.start[worker];
}
template <bool EVEN>
__device__ __forceinline__ int plan_cum(const ChunkPlan& p, int tile) {
  return is_even<EVEN>(p) ? tile * p.even.blocks : p.cum[tile];
}
template <bool EVEN>
__device__ __forceinline__ int4 plan_tile(const ChunkPlan& p, int tile) {
  if (!is_even<EVEN>(p)) return p.tile[tile];
  const int b = tile / p.even.tiles, row = (tile - b * p.even.tiles) * 64;
  return make_int4(b, b * p.even.heads + row, min(64, p.even.heads - row), 0);
}
template <bool EVEN>
__device__ __forceinline__ int plan_len(const ChunkArgs& a, const ChunkPlan& p, int b) {
  return is_even<EVEN>(p) ? a.listed : p.seq_len[b];
}

__device__ __forceinline__ int find_last_le(const int32_t* a, int n, int x) {   // a[0] <= x
  int lo = 0;
  for (int hi = n; hi - lo > 1;) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Visible positions [lo, hi) of token t of sequence b (hi <= lo: none), its position in
// *pos.  len: positions of the sequence that can be seen.  Neither is below 0, so that their
// distance to a block's first position is an int, whatever the masks hold.
__device__ __forceinline__ void visible(const ChunkArgs& a, int b, int t, int len, int* lo, int* hi, int* pos) {
  if (a.listed > 0) {
    *pos = 0;
    *lo = 0;
    *hi = len;
    return;
  }
  *pos = a.kv_lens[b] - (a.cu_q[b + 1] - t);
  *lo = a.vis_begin != nullptr ? max(0, a.vis_begin[t]) : 0;
  *hi = max(0, min(len, a.vis_end != nullptr ? a.vis_end[t] : *pos + 1));
}

// What a sequence brings: its entries of q, clamped to it, and its blocks.  wrong: its offsets
// decrease or are not q's, so that its entries may be another's too, or its positions astray.
struct Sequence {
  int first, n, len, blocks;
  bool wrong;
};
__device__ __forceinline__ Sequence sequence(const ChunkArgs& a, int b) {
  Sequence s = {0, 0, 0, 0, false};
  if (b >= a.B) return s;
  const int c0 = a.cu_q[b], c1 = a.cu_q[b + 1];
  s.wrong = c0 < 0 || c1 < c0 || c1 > a.T;
  s.len = max(a.kv_lens[b], 0);
  s.first = min(max(c0, 0), a.T);
  s.n = min(max(c1, s.first), a.T) - s.first;
  // one without cached tokens keeps one block (of zeros) for its tiles to read; a length may be
  // as large as its type allows (seq_len below cuts it to the copy)
  if (s.n > 0) s.blocks = max(1, s.len / kChunkBlk + (s.len % kChunkBlk != 0 ? 1 : 0));
  return s;
}
// Its first block in the expanded copy, given the blocks before it, and how many positions
// of it find room there.
__device__ __forceinline__ int seq_base(const ChunkPlan& p, long long before) {
  return static_cast<int>(min(before, static_cast<long long>(p.cap_blocks)));
}
__device__ __forceinline__ int seq_len(const ChunkPlan& p, const Sequence& s, long long before) {
  const long long left = p.cap_blocks - before;
  return s.blocks <= left ? s.len : left > 0 ? static_cast<int>(left) * kChunkBlk : 0;
}

// The first block that rows row .. row + rows - 1 of sequence b see, and how many (one at least).
__device__ __forceinline__ void tile_blocks(const ChunkArgs& a, int b, int row, int rows, int len, int* first, int* n) {
  int low = 0x7fffffff, high = 0;
  for (int tok = row / a.H; tok <= (row + rows - 1) / a.H; ++tok) {
    int lo, hi, pos;
    visible(a, b, tok, len, &lo, &hi, &pos);
    if (hi > lo) {
      low = min(low, lo);
      high = max(high, hi);
    }
  }
  *first = high > 0 ? low / kChunkBlk : 0;
  *n = high > 0 ? (high - 1) / kChunkBlk + 1 - *first : 1;
}

// Pair kernel: tiles of 256 rows on pairs of SMs, over the expanded copy.
constexpr int kPairRows = 256;
cudaError_t pair_workers(int* workers);
cudaError_t launch_chunk_pair(const ChunkArgs& a, const ChunkPlan& p, int workers, cudaStream_t stream);

// Single kernel: tiles of 64 rows on one SM each, which expands the rows itself.
constexpr int kSingleRows = 64;
constexpr int kFewTiles = 32;      // a lane each
cudaError_t launch_chunk_single(const ChunkArgs& a, const ChunkPlan& p, int workers, cudaStream_t stream);

// The tensor map of `rows` rows of 512 bf16, in boxes of 64 columns, 128-byte swizzle.
cudaError_t encode_rows(CUtensorMap* map, const void* base, int64_t rows, int box_rows);

}  // namespace smla
