// Ranking of free pages across a planning cluster, and copies of rows within the pool: shared by
// the page calls.
#pragma once
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/smla.h"
#include "smla_internal.h"

namespace smla {

namespace cg = cooperative_groups;

constexpr int kPlanCtas = 8;        // CTAs of the planning cluster (the portable size)
constexpr int kPlanThreads = 1024;

// ---------------------------------------------------------------------------
// Ranking across the planning cluster
// ---------------------------------------------------------------------------
struct PlanShared {
  int warp[32];
  int2 counts[2][kPlanCtas];   // counts of every CTA of the cluster, two slots in turn
};

// Exclusive sum of v over the CTA's threads; *total gets the sum.  All threads call.
__device__ __forceinline__ int block_rank(int v, int* total, PlanShared* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  __syncthreads();            // the previous call's readers are done with warp[]
  if (lane == 31) sh->warp[warp] = s;
  __syncthreads();
  if (warp == 0) {
    int w = sh->warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    sh->warp[lane] = w;
  }
  __syncthreads();
  *total = sh->warp[31];
  return s - v + (warp > 0 ? sh->warp[warp - 1] : 0);
}

// Shares this CTA's two counts with the cluster (a slot may be used again after another
// share): *before = sums of the lower ranks', returns the sums of all.  Orders the
// cluster's memory accesses as a barrier does.
__device__ __forceinline__ int2 cluster_share(int2 mine, int slot, int2* before, PlanShared* sh) {
  cg::cluster_group cl = cg::this_cluster();
  const int rank = static_cast<int>(cl.block_rank());
  if (threadIdx.x < kPlanCtas) cl.map_shared_rank(sh, threadIdx.x)->counts[slot][rank] = mine;
  cl.sync();
  int2 all = make_int2(0, 0), low = make_int2(0, 0);
#pragma unroll
  for (int r = 0; r < kPlanCtas; ++r) {
    const int2 c = sh->counts[slot][r];
    all.x += c.x;
    all.y += c.y;
    if (r < rank) {
      low.x += c.x;
      low.y += c.y;
    }
  }
  *before = low;
  return all;
}

// This CTA's part [first, last) of n things, and within it the thread's part, a run of a
// multiple of 4: ranks then need one block-wide sum, whatever the length.  Unsigned, since the ends
// of a part of nearly 2^31 things are rounded up past it.
struct Part {
  uint32_t run0, run1;
};
__device__ __forceinline__ Part part_of(uint32_t n) {
  const uint32_t rank = cg::this_cluster().block_rank();
  const uint32_t per = ((n + kPlanCtas - 1) / kPlanCtas + 3) & ~3u;
  const uint32_t first = min(n, rank * per), last = min(n, first + per);
  const uint32_t run = ((last - first + kPlanThreads - 1) / kPlanThreads + 3) & ~3u;
  Part p;
  p.run0 = min(last, first + threadIdx.x * run);
  p.run1 = min(last, p.run0 + run);
  return p;
}
// f(page, count) for the pages of the thread's run.
template <class F>
__device__ __forceinline__ void each_page(const int32_t* ref, const Part& p, F f) {
  for (uint32_t q = p.run0; q < p.run1; q += 4) {
    int c[4];
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) c[k] = q + k < p.run1 ? __ldcg(ref + q + k) : 0;
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k)
      if (q + k < p.run1) f(static_cast<int>(q + k), c[k]);
  }
}
__device__ __forceinline__ int count_free(const int32_t* ref, const Part& p) {
  int n = 0;
  each_page(ref, p, [&](int, int c) { n += c <= 0; });
  return n;
}
// Gives the `want` lowest free pages (or all) a count of 1 and lists them, ascending.
// rank: free pages before the thread's run.
__device__ __forceinline__ void take_free(int32_t* ref, const Part& p, int rank, int want, int32_t* list) {
  if (rank >= want) return;
  each_page(ref, p, [&](int page, int c) {
    if (c <= 0) {
      if (rank < want) {
        list[rank] = page;
        ref[page] = 1;
      }
      ++rank;
    }
  });
}

// f(entry) for the entries of a row of the table, by the CTA's threads.  Unsigned, since the count behind
// the last of nearly 2^31 entries is past an int.
template <class F>
__device__ __forceinline__ void each_entry(int max_pages, F f) {
  for (uint32_t e = threadIdx.x; e < static_cast<uint32_t>(max_pages); e += blockDim.x) f(static_cast<int>(e));
}

// Copies rows from .. from + rows - 1 of the pool to to .. by the CTA's threads.  Rows that
// follow one another without a gap go as 16-byte words where both ends allow it, four of a
// thread's in flight.
__device__ __forceinline__ void copy_rows(uint8_t* pool, int64_t stride, int64_t from, int64_t to,
                                          int rows) {
  const int row_bytes = is_row4(stride) ? kRow4Bytes : kRowBytes;
  const uint8_t* s = pool + from * stride;
  uint8_t* d = pool + to * stride;
  if (stride == row_bytes) {
    // 16-byte aligned parts: both start on one, or both 8 bytes behind one
    const bool same = ((reinterpret_cast<uintptr_t>(s) ^ reinterpret_cast<uintptr_t>(d)) & 8) == 0;
    if (same) {
      const int bytes = rows * row_bytes;
      const int head = static_cast<int>(reinterpret_cast<uintptr_t>(s) & 8);
      const int units = (bytes - head) / 16, tail = bytes - head - 16 * units;
      if (threadIdx.x == 0 && head) *reinterpret_cast<uint2*>(d) = *reinterpret_cast<const uint2*>(s);
      if (threadIdx.x == 1 && tail)
        *reinterpret_cast<uint2*>(d + bytes - 8) = *reinterpret_cast<const uint2*>(s + bytes - 8);
      const uint4* s4 = reinterpret_cast<const uint4*>(s + head);
      uint4* d4 = reinterpret_cast<uint4*>(d + head);
      const int step = blockDim.x;
      for (int w = threadIdx.x; w < units; w += 4 * step) {
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (w + k * step < units) v[k] = __ldcs(s4 + w + k * step);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (w + k * step < units) __stcs(d4 + w + k * step, v[k]);
      }
      return;
    }
  }
  const int words = row_bytes / 8;
  for (int w = threadIdx.x; w < rows * words; w += blockDim.x) {
    const int64_t off = (w / words) * stride + 8 * (w % words);
    *reinterpret_cast<uint2*>(d + off) = *reinterpret_cast<const uint2*>(s + off);
  }
}

}  // namespace smla
