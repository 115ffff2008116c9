// What the translation units of the chunk attention share: the arguments of a call, its
// plan in the workspace, and the launches.  Not part of the public ABI.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/smla.h"
#include "smla_internal.h"

namespace smla {

constexpr int kChunkBlk = 64;     // positions of a block

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
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
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
  *pos = a.kv_lens[b] - (a.cu_q[b + 1] - t);
  *lo = a.vis_begin != nullptr ? max(0, a.vis_begin[t]) : 0;
  *hi = max(0, min(len, a.vis_end != nullptr ? a.vis_end[t] : *pos + 1));
}

// Pair kernel: tiles of 256 rows on pairs of SMs, over the expanded copy.
constexpr int kPairRows = 256;
cudaError_t pair_workers(int* workers);
cudaError_t launch_chunk_pair(const ChunkArgs& a, const ChunkPlan& p, int workers, cudaStream_t stream);

// Single kernel: tiles of 64 rows on one SM each, which expands the rows itself.
constexpr int kSingleRows = 64;
cudaError_t launch_chunk_single(const ChunkArgs& a, const ChunkPlan& p, int workers, cudaStream_t stream);

// The tensor map of `rows` rows of 512 bf16, in boxes of 64 columns, 128-byte swizzle.
cudaError_t encode_rows(CUtensorMap* map, const void* base, int64_t rows, int box_rows);

}  // namespace smla
