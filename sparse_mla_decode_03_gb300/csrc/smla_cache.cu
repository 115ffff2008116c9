// The paged cache: quantising new tokens into its rows (smla_cache_append) and managing
// its pages (smla_cache_reserve, _fork, _free, _compact).  Declared and documented in
// include/smla.h.
//
// Page calls.  A page is free exactly when its count is 0, so no free list is kept: a
// call scans the counts.  The scans and the rankings that depend on one another run as
// one thread-block cluster of 8 CTAs (hardware cluster barriers between the phases, a
// CTA's slice of the pages or table each), so a call is one launch, plus one wide launch
// where rows of the cache move.  Page calls are bound by launches and by the trips to memory
// and cluster barriers of a plan: free 4 us, fork 10 + 5.5 (512 children 11 + 8), reserve 6 (of
// 528 rows and 32,768 pages 12.5), compaction's plan 7.5 (32,768 pages 11).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/smla.h"
#include "smla_internal.h"
#include "smla_ptx.cuh"

namespace cg = cooperative_groups;

namespace smla {
namespace {

constexpr int kPlanCtas = 8;        // CTAs of the planning cluster (the portable size)
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ void report(int* status, int code) { atomicCAS(status, 0, code); }

// ---------------------------------------------------------------------------
// Append
// ---------------------------------------------------------------------------
struct AppendArgs {
  const uint4* kv;
  int64_t token_units;    // 16-byte units between tokens
  int total;
  uint8_t* pool;
  const int32_t *table, *cu_q, *kv_lens;
  int B, max_pages, page_size, num_pages;
  int64_t stride;
  int* status;
};

// Sequence of token t: the warp narrows [0, B) 32-fold a step.  -1 outside every one.
__device__ __forceinline__ int sequence_of(const int32_t* cu_q, int B, int t) {
  if (t < __ldg(cu_q) || t >= __ldg(cu_q + B)) return -1;
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B;     // cu_q[lo] <= t < cu_q[hi]
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + (lane + 1) * step;
    const bool below = at < hi && __ldg(cu_q + at) <= t;
    const int k = __popc(__ballot_sync(0xffffffffu, below));
    lo += k * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// The row of token t, or null (reported) if it has no place; null too outside every sequence.
__device__ __forceinline__ uint8_t* row_of(const AppendArgs& a, int t) {
  const int b = sequence_of(a.cu_q, a.B, t);
  if (b < 0) return nullptr;
  const int64_t pos = static_cast<int64_t>(__ldg(a.kv_lens + b)) - (__ldg(a.cu_q + b + 1) - t);
  if (pos >= 0) {   // below 2^31: kv_lens is an int32
    const uint32_t at = static_cast<uint32_t>(pos), page = at / static_cast<uint32_t>(a.page_size);
    if (page < static_cast<uint32_t>(a.max_pages)) {
      const int phys = __ldg(a.table + static_cast<int64_t>(b) * a.max_pages + page);
      if (phys >= 0 && phys < a.num_pages)
        return a.pool + (static_cast<int64_t>(phys) * a.page_size + (at - page * a.page_size)) * a.stride;
    }
  }
  if ((threadIdx.x & 31) == 0) report(a.status, SMLA_ERR_INDEX_RANGE);
  return nullptr;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// One token of a warp.  Lane l < 28 holds nope columns 16 l .. 16 l + 15 (four lanes a scale
// group), lanes 28..31 the rope.  The row is put together in shared memory (stage: 73 words)
// and leaves in consecutive words.
__device__ __forceinline__ void write_row(const AppendArgs& a, uint8_t* dst, const uint4& u0, const uint4& u1,
                                          uint2* stage) {
  const int lane = threadIdx.x & 31;
  uint32_t w[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
  // largest magnitude as bf16 bits, two columns at a time (magnitudes compare as integers)
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_u16x2(m, w[i] & 0x7fff7fffu);
  uint32_t top = max(m >> 16, m & 0xffffu);
  if (__any_sync(0xffffffffu, lane < 28 && top >= 0x7f80u)) {
    // infinity and NaN are stored as NaN and do not count
    top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t h[2] = {w[i] & 0xffffu, w[i] >> 16};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if ((h[k] & 0x7fffu) >= 0x7f80u) {
          h[k] = 0x7fffu;
          if (lane < 28) report(a.status, SMLA_ERR_RANGE);
        } else {
          top = max(top, h[k] & 0x7fffu);
        }
      }
      w[i] = h[0] | h[1] << 16;
    }
  }
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  // 448 = 1.75 * 2^8, so the least e with top <= 448 * 2^e follows from top's exponent
  // and whether its mantissa exceeds 1.75: exact, no logarithm.
  int byte = static_cast<int>(top >> 7) - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0);
  byte = top == 0 ? 127 : min(max(byte, 1), 254);
  // from 1.9375 * 2^127 on (halfway from 240 to 256 in the scale 2^120) the stored value is 2^128
  if (top >= 0x7f78u && lane < 28) report(a.status, SMLA_ERR_RANGE);
  // 2^(127 - byte) as a float (byte 254: the subnormal 2^-127)
  const float inv = __uint_as_float(byte < 254 ? static_cast<uint32_t>(254 - byte) << 23 : 0x00400000u);
  if (lane < 28) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint16_t lo, hi;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
          : "=h"(lo)
          : "f"(__uint_as_float(w[2 * i] & 0xffff0000u) * inv), "f"(__uint_as_float(w[2 * i] << 16) * inv));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
          : "=h"(hi)
          : "f"(__uint_as_float(w[2 * i + 1] & 0xffff0000u) * inv), "f"(__uint_as_float(w[2 * i + 1] << 16) * inv));
      o[i] = lo | (static_cast<uint32_t>(hi) << 16);
    }
    stage[2 * lane] = make_uint2(o[0], o[1]);
    stage[2 * lane + 1] = make_uint2(o[2], o[3]);
    if ((lane & 3) == 0) reinterpret_cast<uint8_t*>(stage)[kNope + lane / 4] = static_cast<uint8_t>(byte);
  } else {
    uint2* d = stage + 57 + 4 * (lane - 28);
    d[0] = make_uint2(u0.x, u0.y);
    d[1] = make_uint2(u0.z, u0.w);
    d[2] = make_uint2(u1.x, u1.y);
    d[3] = make_uint2(u1.z, u1.w);
    if (lane == 28) reinterpret_cast<uint8_t*>(stage)[kNope + 7] = 0;      // the padding
  }
  __syncwarp();
  uint2* d = reinterpret_cast<uint2*>(dst);
  d[lane] = stage[lane];
  d[lane + 32] = stage[lane + 32];
  if (lane < 9) d[lane + 64] = stage[lane + 64];
  __syncwarp();
}

// Bound by memory: 1,024 bytes in and 584 out a token.  One token a warp: 38 us for 131,072 tokens
// (5.55 TB/s, 82 % of the measured copy rate; issue 73 %, integer pipe 59 % busy); two or four
// tokens' loads at once measured 41.0 and 44.1 us.  A decode step's call (96 tokens) is a launch
// and two trips to memory, 5 us.
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs a) {
  __shared__ uint2 stage[8][76];
  grid_dep_wait();
  grid_dep_launch();
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= a.total) return;
  const uint4* src = a.kv + t * a.token_units + 2 * (threadIdx.x & 31);
  const uint4 u0 = __ldcs(src), u1 = __ldcs(src + 1);
  uint8_t* dst = row_of(a, t);
  if (dst != nullptr) write_row(a, dst, u0, u1, stage[threadIdx.x >> 5]);
}

// ---------------------------------------------------------------------------
// Ranking across the planning cluster
// ---------------------------------------------------------------------------
struct PlanShared {
  int warp[32];
  int2 counts[2][kPlanCtas];   // counts of every CTA of the cluster, two slots in turn
};

// Exclusive sum of v over the CTA's threads; *total gets the sum.  All threads call.
__device__ int block_rank(int v, int* total, PlanShared* sh) {
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
__device__ int2 cluster_share(int2 mine, int slot, int2* before, PlanShared* sh) {
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

// ---------------------------------------------------------------------------
// Reserve
// ---------------------------------------------------------------------------
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
    reserve_kernel(int32_t* ref, int32_t* table, const int32_t* target, int rows, int max_pages,
                   int page_size, int num_pages, int32_t* list, int* status) {
  __shared__ PlanShared sh;
  cg::this_cluster().sync();   // every CTA has started: its shared memory may be written
  grid_dep_wait();
  grid_dep_launch();
  // The table row after row: each CTA a part, each thread a run of it, so that a rank is the
  // entries before the run plus those in it.
  const Part pp = part_of(num_pages);
  const int64_t entries = static_cast<int64_t>(rows) * max_pages;
  const int64_t per = (entries + kPlanCtas - 1) / kPlanCtas;
  const int64_t first = min(entries, cg::this_cluster().block_rank() * per), last = min(entries, first + per);
  const int64_t run = (last - first + kPlanThreads - 1) / kPlanThreads;
  const int64_t run0 = min(last, first + threadIdx.x * run), run1 = min(last, run0 + run);
  // f(entry) for the unmapped entries of the run that the targets need
  auto each_open = [&](auto f) {
    int r = static_cast<int>(run0 / max_pages), c = static_cast<int>(run0 - static_cast<int64_t>(r) * max_pages);
    int64_t i = run0;
    while (i < run1) {
      const int len = __ldg(target + r);
      int need = len > 0 ? (len - 1) / page_size + 1 : 0;
      if (need > max_pages) {
        if (c == 0) report(status, SMLA_ERR_INDEX_RANGE);
        need = max_pages;
      }
      const int64_t row_end = min(run1, i - c + max_pages), stop = min(run1, i - c + need);
      int32_t* e = table;
#pragma unroll 4
      for (; i < stop; ++i)
        if (__ldcg(e + i) < 0) f(i);
      i = row_end;
      ++r;
      c = 0;
    }
  };
  int free_total, need_total, mine = 0;
  const int free_rank = block_rank(count_free(ref, pp), &free_total, &sh);
  each_open([&](int64_t) { ++mine; });
  const int need_rank = block_rank(mine, &need_total, &sh);
  int2 low;
  const int2 all = cluster_share(make_int2(need_total, free_total), 0, &low, &sh);
  const int got = min(all.x, all.y);
  take_free(ref, pp, low.y + free_rank, got, list);
  if (all.x > got && blockIdx.x == 0 && threadIdx.x == 0) report(status, SMLA_ERR_POOL_EXHAUSTED);
  if (got == 0) return;
  cg::this_cluster().sync();
  int k = low.x + need_rank;
  if (mine > 0 && k < got)
    each_open([&](int64_t i) {
      if (k < got) table[i] = __ldcg(list + k);
      ++k;
    });
}

// ---------------------------------------------------------------------------
// Fork
// ---------------------------------------------------------------------------
struct ForkArgs {
  uint8_t* pool;
  int32_t *ref, *table, *kv_lens;
  const int32_t *parents, *children;
  int32_t *list, *fresh;      // workspace: free pages taken; the new page of each pair
  int n, rows, max_pages, page_size, num_pages;
  int64_t stride;
  int* status;
};
constexpr int kNoPage = -1, kNotNeeded = -2, kSkip = -3;

// The pair's parent length, or -1 if the pair is to be skipped.
__device__ __forceinline__ int fork_length(const ForkArgs& a, int i) {
  const int p = __ldg(a.parents + i), c = __ldg(a.children + i);
  if (p < 0 || p >= a.rows || c < 0 || c >= a.rows || p == c) return -1;
  const int len = a.kv_lens[p];
  return len < 0 || len > static_cast<int64_t>(a.max_pages) * a.page_size ? -1 : len;
}

// Whether the child of a parent of `len` tokens gets a page of its own: the last one is partly
// filled, and mapped (an entry that names no page of the pool is copied as it is).
__device__ __forceinline__ bool fork_takes(const ForkArgs& a, int i, int len) {
  if (len <= 0 || len % a.page_size == 0) return false;
  const int page = a.table[static_cast<int64_t>(__ldg(a.parents + i)) * a.max_pages + len / a.page_size];
  return page >= 0 && page < a.num_pages;
}

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
    fork_plan_kernel(const ForkArgs a) {
  __shared__ PlanShared sh;
  cg::this_cluster().sync();   // every CTA has started: its shared memory may be written
  grid_dep_wait();
  grid_dep_launch();
  const Part ip = part_of(a.n), pp = part_of(a.num_pages);
  int free_total, need_total, mine = 0;
  const int free_rank = block_rank(count_free(a.ref, pp), &free_total, &sh);
  for (int i = static_cast<int>(ip.run0); i < static_cast<int>(ip.run1); ++i) {
    mine += fork_takes(a, i, fork_length(a, i));
  }
  const int need_rank = block_rank(mine, &need_total, &sh);
  int2 low;
  const int2 all = cluster_share(make_int2(need_total, free_total), 0, &low, &sh);
  const int got = min(all.x, all.y);
  take_free(a.ref, pp, low.y + free_rank, got, a.list);
  cg::this_cluster().sync();
  int k = low.x + need_rank;
  for (int i = static_cast<int>(ip.run0); i < static_cast<int>(ip.run1); ++i) {
    const int len = fork_length(a, i);
    int f = len < 0 ? kSkip : kNotNeeded;
    if (fork_takes(a, i, len)) {
      f = k < got ? __ldcg(a.list + k) : kNoPage;
      ++k;
    }
    if (f == kSkip) report(a.status, SMLA_ERR_INDEX_RANGE);
    if (f == kNoPage) report(a.status, SMLA_ERR_POOL_EXHAUSTED);
    a.fresh[i] = f;
  }
}

// Copies rows from .. from + rows - 1 of the pool to to .. by the CTA's threads.  Rows that
// follow one another without a gap go as 16-byte words where both ends allow it, four of a
// thread's in flight.
__device__ __forceinline__ void copy_rows(uint8_t* pool, int64_t stride, int64_t from, int64_t to,
                                          int rows) {
  const uint8_t* s = pool + from * stride;
  uint8_t* d = pool + to * stride;
  if (stride == kRowBytes) {
    // 16-byte aligned parts: both start on one, or both 8 bytes behind one
    const bool same = ((reinterpret_cast<uintptr_t>(s) ^ reinterpret_cast<uintptr_t>(d)) & 8) == 0;
    if (same) {
      const int bytes = rows * kRowBytes;
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
  for (int w = threadIdx.x; w < rows * (kRowBytes / 8); w += blockDim.x) {
    const int64_t off = (w / (kRowBytes / 8)) * stride + 8 * (w % (kRowBytes / 8));
    *reinterpret_cast<uint2*>(d + off) = *reinterpret_cast<const uint2*>(s + off);
  }
}

constexpr int kForkRows = 16;   // rows of a partial page that one CTA copies

// Grid (pairs, row groups of a page): group 0 also writes the child's table row.
__global__ void __launch_bounds__(256) fork_apply_kernel(const ForkArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int i = blockIdx.x;
  const int fresh = a.fresh[i];
  if (fresh == kSkip) return;
  const int p = a.parents[i], c = a.children[i];
  const int len = fresh == kNoPage ? 0 : a.kv_lens[p];
  const int full = len / a.page_size, rem = len % a.page_size;
  const int32_t* src = a.table + static_cast<int64_t>(p) * a.max_pages;
  if (blockIdx.y == 0) {
    int32_t* dst = a.table + static_cast<int64_t>(c) * a.max_pages;
    for (int e = threadIdx.x; e < a.max_pages; e += blockDim.x) {
      int v = -1;
      if (e < full) {
        v = src[e];
      } else if (e == full && rem > 0) {
        v = fresh >= 0 ? fresh : src[e];
      }
      if (v >= a.num_pages) report(a.status, SMLA_ERR_INDEX_RANGE);
      else if (v >= 0 && e < full) atomicAdd(a.ref + v, 1);
      dst[e] = v;
    }
    if (threadIdx.x == 0) a.kv_lens[c] = len;
  }
  if (fresh < 0 || rem == 0) return;
  const int from = src[full];
  if (from < 0 || from >= a.num_pages) return;
  for (int r0 = blockIdx.y * kForkRows; r0 < rem; r0 += gridDim.y * kForkRows) {
    copy_rows(a.pool, a.stride, static_cast<int64_t>(from) * a.page_size + r0,
                static_cast<int64_t>(fresh) * a.page_size + r0, min(kForkRows, rem - r0));
  }
}

// ---------------------------------------------------------------------------
// Free
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256)
    free_kernel(int32_t* ref, int32_t* table, int32_t* kv_lens, const int32_t* rows, int num_rows,
                int max_pages, int num_pages, int* status) {
  grid_dep_wait();
  grid_dep_launch();
  const int r = __ldg(rows + blockIdx.x);
  if (r < 0 || r >= num_rows) {
    if (threadIdx.x == 0) report(status, SMLA_ERR_INDEX_RANGE);
    return;
  }
  int32_t* e = table + static_cast<int64_t>(r) * max_pages;
  for (int i = threadIdx.x; i < max_pages; i += blockDim.x) {
    if (e[i] < 0) continue;
    const int p = atomicExch(e + i, -1);   // a row listed twice gives its pages back once
    if (p < 0) continue;
    if (p >= num_pages) {
      report(status, SMLA_ERR_INDEX_RANGE);
    } else if (atomicSub(ref + p, 1) <= 0) {
      atomicAdd(ref + p, 1);
      report(status, SMLA_ERR_INDEX_RANGE);
    }
  }
  if (threadIdx.x == 0) kv_lens[r] = 0;
}

// ---------------------------------------------------------------------------
// Compact
// ---------------------------------------------------------------------------
struct CompactArgs {
  uint8_t* pool;
  const int32_t *ref, *table;
  int32_t *ref_out, *table_out, *info;
  int32_t *movers, *holes, *rank_of;   // workspace
  int64_t entries;
  int page_size, num_pages;
  int64_t stride;
  int* status;
};

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
    compact_plan_kernel(const CompactArgs a) {
  __shared__ PlanShared sh;
  cg::this_cluster().sync();   // every CTA has started: its shared memory may be written
  grid_dep_wait();
  grid_dep_launch();
  const Part pp = part_of(a.num_pages);
  int mine = 0, total;
  each_page(a.ref, pp, [&](int, int c) { mine += c > 0; });
  const int rank = block_rank(mine, &total, &sh);
  int2 low;
  const int used = cluster_share(make_int2(total, 0), 0, &low, &sh).x;
  // Holes are the free pages below `used`, movers the pages in use at or past it.  With r
  // pages in use below page p, p - r free ones are: a hole's rank; a mover's is r less the
  // pages in use below `used`, which the second share counts.  rank_of tells the table's entries
  // apart: the rank of a mover, -1 of a page that nobody owns, 0 of one that stays.
  int r = low.x + rank, kept_here = 0;
  each_page(a.ref, pp, [&](int p, int c) {
    if (p < used) {
      if (c <= 0) a.holes[p - r] = p;
      else ++kept_here;
      a.rank_of[p] = c > 0 ? 0 : -1;
    } else {
      a.rank_of[p] = c > 0 ? r : -1;
    }
    r += c > 0;
  });
  block_rank(kept_here, &total, &sh);
  const int kept = cluster_share(make_int2(total, 0), 1, &low, &sh).x;
  const int moved = used - kept;
  // counts: each thread of a move reads and writes both of its pages' counts itself, so
  // ref_out may be ref
  each_page(a.ref, pp, [&](int p, int c) {
    if (p < used) {
      if (c > 0) a.ref_out[p] = c;
    } else if (c > 0) {
      const int k = __ldcg(a.rank_of + p) - kept;
      a.movers[k] = p;
      a.ref_out[__ldcg(a.holes + k)] = c;
      a.ref_out[p] = 0;
    } else {
      a.ref_out[p] = c;
    }
  });
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.info[0] = used;
    a.info[1] = moved;
  }
}

// Rewrites the table and moves the listed pages: a CTA takes chunks of kMoveRows rows in turn.  Bound by memory: 7,889
// pages of 64 rows, 37 KB each in and out, in 87 us, the measured copy rate.
constexpr int kMoveRows = 28;      // 16,352 bytes: four 16-byte words a thread
__global__ void __launch_bounds__(256) compact_move_kernel(const CompactArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int used = a.info[0], moved = a.info[1], kept = used - moved;
  // the table, each entry by itself
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < a.entries; i += step) {
    int v = a.table[i];
    if (v >= a.num_pages) {
      report(a.status, SMLA_ERR_INDEX_RANGE);
    } else if (v >= 0) {
      const int r = a.rank_of[v];
      if (r < 0) report(a.status, SMLA_ERR_INDEX_RANGE);
      else if (v >= used) v = a.holes[r - kept];
    }
    a.table_out[i] = v;
  }
  const int per = (a.page_size + kMoveRows - 1) / kMoveRows;
  const int64_t chunks = static_cast<int64_t>(moved) * per;
  for (int64_t i = blockIdx.x; i < chunks; i += gridDim.x) {
    const int k = static_cast<int>(i / per), r0 = static_cast<int>(i % per) * kMoveRows;
    copy_rows(a.pool, a.stride, static_cast<int64_t>(a.movers[k]) * a.page_size + r0,
              static_cast<int64_t>(a.holes[k]) * a.page_size + r0, min(kMoveRows, a.page_size - r0));
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int check_cache(const smla_cache_params* c) {
  if (c == nullptr || c->num_pages < 1 || c->page_size < 1 || c->num_seqs < 1 || c->max_pages < 1)
    return SMLA_ERR_INVALID_ARG;
  if (c->kv_row_stride < kRowBytes || c->kv_row_stride % 8 != 0) return SMLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(c->num_pages) * c->page_size > (int64_t{1} << 31) || c->num_seqs > 65535)
    return SMLA_ERR_UNSUPPORTED_SHAPE;
  return SMLA_OK;
}

bool ints_ok(const void* p) { return p != nullptr && aligned(p, 4); }
bool pool_ok(const void* p) { return p != nullptr && aligned(p, 8); }

// Workspace: three lists of num_pages entries, one of num_seqs.
size_t list_bytes(const smla_cache_params* c) { return round256(size_t{4} * c->num_pages); }

int check_workspace(const smla_cache_params* c, const void* ws, size_t bytes) {
  if (ws == nullptr || !aligned(ws, 256)) return SMLA_ERR_INVALID_ARG;
  size_t need = 0;
  const int st = smla_cache_workspace_size(c, &need);
  if (st != SMLA_OK) return st;
  return bytes < need ? SMLA_ERR_WORKSPACE_TOO_SMALL : SMLA_OK;
}

// The device check and the status word; the last step before a launch.
int ready(int** status) {
  const int st = check_device();
  if (st != SMLA_OK) return st;
  return status_word_address(status) == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

int done(cudaError_t e) { return e == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA; }

}  // namespace
}  // namespace smla

using namespace smla;   // NOLINT: the entry points below are this file's own

extern "C" {

int smla_cache_append(const void* kv, int64_t kv_token_stride, int32_t total_tokens, void* kv_pages,
                      const int32_t* block_table, const int32_t* cu_q, const int32_t* kv_lens,
                      const smla_cache_params* c, smla_stream_t stream) {
  int st = check_cache(c);
  if (st != SMLA_OK) return st;
  if (total_tokens < 0 || kv_token_stride < kQkDim || kv_token_stride % 8 != 0)
    return SMLA_ERR_INVALID_ARG;
  if (!pool_ok(kv_pages) || !ints_ok(block_table) || !ints_ok(cu_q) || !ints_ok(kv_lens))
    return SMLA_ERR_INVALID_ARG;
  if (total_tokens == 0) return SMLA_OK;
  if (kv == nullptr || !aligned(kv, 16)) return SMLA_ERR_INVALID_ARG;
  int* status = nullptr;
  st = ready(&status);
  if (st != SMLA_OK) return st;
  const AppendArgs a = {static_cast<const uint4*>(kv), kv_token_stride / 8, total_tokens,
                        static_cast<uint8_t*>(kv_pages), block_table, cu_q, kv_lens, c->num_seqs,
                        c->max_pages, c->page_size, c->num_pages, c->kv_row_stride, status};
  return done(launch_programmatic(append_kernel, dim3((total_tokens - 1) / 8 + 1), dim3(256), 0,
                                  reinterpret_cast<cudaStream_t>(stream), a));
}

int smla_cache_workspace_size(const smla_cache_params* c, size_t* bytes) {
  const int st = check_cache(c);
  if (st != SMLA_OK) return st;
  if (bytes == nullptr) return SMLA_ERR_INVALID_ARG;
  *bytes = 3 * list_bytes(c) + round256(size_t{4} * c->num_seqs);
  return SMLA_OK;
}

int smla_cache_reserve(int32_t* ref_count, int32_t* block_table, const int32_t* target_lens,
                       const smla_cache_params* c, void* workspace, size_t workspace_bytes,
                       smla_stream_t stream) {
  int st = check_cache(c);
  if (st != SMLA_OK) return st;
  if (!ints_ok(ref_count) || !ints_ok(block_table) || !ints_ok(target_lens)) return SMLA_ERR_INVALID_ARG;
  // entries that want a page are counted in ints
  if (static_cast<int64_t>(c->num_seqs) * c->max_pages >= (int64_t{1} << 31)) return SMLA_ERR_UNSUPPORTED_SHAPE;
  st = check_workspace(c, workspace, workspace_bytes);
  if (st != SMLA_OK) return st;
  int* status = nullptr;
  st = ready(&status);
  if (st != SMLA_OK) return st;
  char* ws = static_cast<char*>(workspace);
  return done(launch_programmatic(reserve_kernel, dim3(kPlanCtas), dim3(kPlanThreads), 0,
                                  reinterpret_cast<cudaStream_t>(stream), ref_count, block_table,
                                  target_lens, c->num_seqs, c->max_pages, c->page_size, c->num_pages,
                                  reinterpret_cast<int32_t*>(ws), status));
}

int smla_cache_fork(void* kv_pages, int32_t* ref_count, int32_t* block_table, int32_t* kv_lens,
                    const int32_t* parents, const int32_t* children, int32_t n,
                    const smla_cache_params* c, void* workspace, size_t workspace_bytes,
                    smla_stream_t stream) {
  int st = check_cache(c);
  if (st != SMLA_OK) return st;
  if (n < 0 || n > c->num_seqs) return SMLA_ERR_INVALID_ARG;
  if (!pool_ok(kv_pages) || !ints_ok(ref_count) || !ints_ok(block_table) || !ints_ok(kv_lens))
    return SMLA_ERR_INVALID_ARG;
  st = check_workspace(c, workspace, workspace_bytes);
  if (st != SMLA_OK) return st;
  if (n == 0) return SMLA_OK;
  if (!ints_ok(parents) || !ints_ok(children)) return SMLA_ERR_INVALID_ARG;
  int* status = nullptr;
  st = ready(&status);
  if (st != SMLA_OK) return st;
  char* ws = static_cast<char*>(workspace);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const ForkArgs a = {static_cast<uint8_t*>(kv_pages), ref_count, block_table, kv_lens, parents, children,
                      reinterpret_cast<int32_t*>(ws), reinterpret_cast<int32_t*>(ws + 3 * list_bytes(c)),
                      n, c->num_seqs, c->max_pages, c->page_size, c->num_pages, c->kv_row_stride, status};
  st = done(launch_programmatic(fork_plan_kernel, dim3(kPlanCtas), dim3(kPlanThreads), 0, s, a));
  if (st != SMLA_OK) return st;
  const int groups = (c->page_size - 1) / kForkRows + 1;
  return done(launch_programmatic(fork_apply_kernel, dim3(n, groups < 64 ? groups : 64), dim3(256), 0, s, a));
}

int smla_cache_free(int32_t* ref_count, int32_t* block_table, int32_t* kv_lens, const int32_t* rows,
                    int32_t n, const smla_cache_params* c, smla_stream_t stream) {
  int st = check_cache(c);
  if (st != SMLA_OK) return st;
  if (n < 0 || !ints_ok(ref_count) || !ints_ok(block_table) || !ints_ok(kv_lens)) return SMLA_ERR_INVALID_ARG;
  if (n == 0) return SMLA_OK;
  if (!ints_ok(rows)) return SMLA_ERR_INVALID_ARG;
  int* status = nullptr;
  st = ready(&status);
  if (st != SMLA_OK) return st;
  return done(launch_programmatic(free_kernel, dim3(n), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream),
                                  ref_count, block_table, kv_lens, rows, c->num_seqs, c->max_pages,
                                  c->num_pages, status));
}

int smla_cache_compact(void* kv_pages, const int32_t* ref_count, const int32_t* block_table,
                       int32_t* ref_count_out, int32_t* block_table_out, int32_t* info,
                       const smla_cache_params* c, void* workspace, size_t workspace_bytes,
                       smla_stream_t stream) {
  int st = check_cache(c);
  if (st != SMLA_OK) return st;
  if (!pool_ok(kv_pages) || !ints_ok(ref_count) || !ints_ok(block_table) || !ints_ok(ref_count_out) ||
      !ints_ok(block_table_out) || !ints_ok(info))
    return SMLA_ERR_INVALID_ARG;
  st = check_workspace(c, workspace, workspace_bytes);
  if (st != SMLA_OK) return st;
  int* status = nullptr;
  st = ready(&status);
  if (st != SMLA_OK) return st;
  char* ws = static_cast<char*>(workspace);
  const size_t list = list_bytes(c);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const CompactArgs a = {static_cast<uint8_t*>(kv_pages), ref_count, block_table, ref_count_out,
                         block_table_out, info, reinterpret_cast<int32_t*>(ws),
                         reinterpret_cast<int32_t*>(ws + list), reinterpret_cast<int32_t*>(ws + 2 * list),
                         static_cast<int64_t>(c->num_seqs) * c->max_pages, c->page_size, c->num_pages,
                         c->kv_row_stride, status};
  st = done(launch_programmatic(compact_plan_kernel, dim3(kPlanCtas), dim3(kPlanThreads), 0, s, a));
  if (st != SMLA_OK) return st;
  return done(launch_programmatic(compact_move_kernel, dim3(152 * 8), dim3(256), 0, s, a));
}

}  // extern "C"
