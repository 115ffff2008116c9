// The paged cache: quantising new tokens into its rows (smla_cache_append) and managing
// its pages (smla_cache_reserve, _fork, _free, _compact).  Declared and documented in
// include/smla.h.
//
// Page calls.  A page is free exactly when its count is 0, so no free list is kept: a
// call scans the counts.  The scans and the rankings that depend on one another run as
// one thread-block cluster of 8 CTAs (hardware cluster barriers between the phases, a
// CTA's slice of the pages or table each), so a call is one launch, plus one wide launch
// where rows of the cache move.
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

// One warp a token.  Lane l < 28 holds nope columns 16 l .. 16 l + 15 (four lanes a
// scale group), lanes 28..31 the rope.
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= a.total) return;
  const uint4* src = a.kv + t * a.token_units + 2 * lane;
  const uint4 u0 = __ldg(src), u1 = __ldg(src + 1);
  const int b = sequence_of(a.cu_q, a.B, t);
  if (b < 0) return;
  const int64_t pos = static_cast<int64_t>(__ldg(a.kv_lens + b)) - (__ldg(a.cu_q + b + 1) - t);
  int64_t row = -1;
  if (pos >= 0) {   // below 2^31: kv_lens is an int32
    const uint32_t at = static_cast<uint32_t>(pos), page = at / static_cast<uint32_t>(a.page_size);
    if (page < static_cast<uint32_t>(a.max_pages)) {
      const int phys = __ldg(a.table + static_cast<int64_t>(b) * a.max_pages + page);
      if (phys >= 0 && phys < a.num_pages)
        row = static_cast<int64_t>(phys) * a.page_size + (at - page * a.page_size);
    }
  }
  if (row < 0) {
    if (lane == 0) report(a.status, SMLA_ERR_INDEX_RANGE);
    return;
  }
  uint8_t* dst = a.pool + row * a.stride;
  const uint32_t w[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
  float x[16];
  float top = 0.f;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float m = fabsf(x[i]);
    if (m < INFINITY) {
      top = fmaxf(top, m);
    } else {
      bad = true;
      x[i] = __uint_as_float(0x7fffffffu);   // infinity and NaN are stored as NaN
    }
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  // 448 = 1.75 * 2^8, so the least e with top <= 448 * 2^e follows from top's exponent
  // and whether its mantissa exceeds 1.75: exact, no logarithm.
  const uint32_t tb = __float_as_uint(top);
  int byte = static_cast<int>(tb >> 23) - 8 + ((tb & 0x7fffffu) > 0x600000u ? 1 : 0);
  byte = top == 0.f ? 127 : min(max(byte, 1), 254);
  // 2^(127 - byte) as a float (byte 254: the subnormal 2^-127)
  const float inv = __uint_as_float(byte < 254 ? static_cast<uint32_t>(254 - byte) << 23 : 0x00400000u);
  if (lane < 28) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint16_t lo, hi;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[4 * i + 1] * inv), "f"(x[4 * i] * inv));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[4 * i + 3] * inv), "f"(x[4 * i + 2] * inv));
      o[i] = lo | (static_cast<uint32_t>(hi) << 16);
    }
    uint2* d = reinterpret_cast<uint2*>(dst + 16 * lane);
    d[0] = make_uint2(o[0], o[1]);
    d[1] = make_uint2(o[2], o[3]);
    if (bad) report(a.status, SMLA_ERR_RANGE);
  } else {
    uint2* d = reinterpret_cast<uint2*>(dst + 456 + 32 * (lane - 28));
    d[0] = make_uint2(u0.x, u0.y);
    d[1] = make_uint2(u0.z, u0.w);
    d[2] = make_uint2(u1.x, u1.y);
    d[3] = make_uint2(u1.z, u1.w);
  }
  // the 7 scale bytes and the padding as one 8-byte word
  uint32_t slo = 0, shi = 0;
#pragma unroll
  for (int g = 0; g < 7; ++g) {
    const uint32_t v = static_cast<uint32_t>(__shfl_sync(0xffffffffu, byte, 4 * g));
    if (g < 4) slo |= v << (8 * g);
    else shi |= v << (8 * (g - 4));
  }
  if (lane == 0) *reinterpret_cast<uint2*>(dst + kNope) = make_uint2(slo, shi);
}

// ---------------------------------------------------------------------------
// Ranking across the planning cluster
// ---------------------------------------------------------------------------
struct PlanShared {
  int warp[32];
  int counts[2][kPlanCtas];   // one count of every CTA of the cluster, two in turn
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

// Shares this CTA's count with the cluster (slot 0 or 1; a slot may be used again after
// another share): *before = sum of the lower ranks', returns the sum of all.  Orders
// the cluster's memory accesses as a barrier does.
__device__ int cluster_share(int mine, int slot, int* before, PlanShared* sh) {
  cg::cluster_group cl = cg::this_cluster();
  const int rank = static_cast<int>(cl.block_rank());
  if (threadIdx.x < kPlanCtas) cl.map_shared_rank(sh, threadIdx.x)->counts[slot][rank] = mine;
  cl.sync();
  int all = 0, low = 0;
#pragma unroll
  for (int r = 0; r < kPlanCtas; ++r) {
    const int c = sh->counts[slot][r];
    all += c;
    if (r < rank) low += c;
  }
  *before = low;
  return all;
}

__device__ __forceinline__ void slice(int n, int* first, int* last) {
  const int rank = static_cast<int>(cg::this_cluster().block_rank());
  const int per = ((n + kPlanCtas - 1) / kPlanCtas + 3) & ~3;
  *first = min(n, rank * per);
  *last = min(n, *first + per);
}

// Free pages (in use: inv) of [first, last), this CTA's total.
__device__ int count_pages(const int32_t* ref, int first, int last, bool used, PlanShared* sh) {
  int c = 0;
  for (int p = first + threadIdx.x; p < last; p += kPlanThreads) c += (__ldcg(ref + p) > 0) == used;
  int total;
  block_rank(c, &total, sh);
  return total;
}

// Gives the `want` lowest free pages (fewer where there are not so many) a count of 1
// and lists them, ascending, in `list`.  Returns how many are listed.  Whole cluster.
__device__ int take_free(int32_t* ref, int num_pages, int want, int32_t* list, int slot, PlanShared* sh) {
  int first, last, before;
  slice(num_pages, &first, &last);
  const int mine = want > 0 ? count_pages(ref, first, last, false, sh) : 0;
  const int all = cluster_share(mine, slot, &before, sh);
  const int end = min(want, all);
  for (int at = first; at < last && before < end; at += kPlanThreads) {
    const int p = at + static_cast<int>(threadIdx.x);
    const bool free = p < last && __ldcg(ref + p) <= 0;
    int total;
    const int r = before + block_rank(free ? 1 : 0, &total, sh);
    if (free && r < end) {
      list[r] = p;
      ref[p] = 1;
    }
    before += total;
  }
  cg::this_cluster().sync();
  return end;
}

// ---------------------------------------------------------------------------
// Reserve
// ---------------------------------------------------------------------------
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
    reserve_kernel(int32_t* ref, int32_t* table, const int32_t* target, int rows, int max_pages,
                   int page_size, int num_pages, int32_t* list, int32_t* row_base, int* status) {
  __shared__ PlanShared sh;
  cg::this_cluster().sync();   // every CTA has started: its shared memory may be written
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int first, last;
  slice(rows, &first, &last);
  auto entries = [&](int r) {      // entries of row r that the target needs
    const int len = __ldg(target + r);
    const int64_t need = len > 0 ? (static_cast<int64_t>(len) + page_size - 1) / page_size : 0;
    if (need > max_pages) {
      if (lane == 0) report(status, SMLA_ERR_INDEX_RANGE);
      return max_pages;
    }
    return static_cast<int>(need);
  };
  // unmapped entries of each row of the slice, then their exclusive sums
  int mine = 0;
  for (int r = first + warp; r < last; r += 32) {
    const int need = entries(r);
    const int32_t* e = table + static_cast<int64_t>(r) * max_pages;
    int c = 0;
    for (int i = lane; i < need; i += 32) c += e[i] < 0;
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0) row_base[r] = c;
  }
  __syncthreads();
  for (int at = first; at < last; at += kPlanThreads) {
    const int r = at + static_cast<int>(threadIdx.x);
    const int c = r < last ? row_base[r] : 0;
    int total;
    const int base = mine + block_rank(c, &total, &sh);
    if (r < last) row_base[r] = base;
    mine += total;
  }
  int before;
  const int want = cluster_share(mine, 0, &before, &sh);
  const int got = take_free(ref, num_pages, want, list, 1, &sh);
  if (want > got && threadIdx.x == 0) report(status, SMLA_ERR_POOL_EXHAUSTED);
  for (int r = first + warp; r < last; r += 32) {
    const int need = entries(r);
    int32_t* e = table + static_cast<int64_t>(r) * max_pages;
    int rank = before + row_base[r];
    for (int i0 = 0; i0 < need; i0 += 32) {
      const int i = i0 + lane;
      const bool open = i < need && e[i] < 0;
      const uint32_t mask = __ballot_sync(0xffffffffu, open);
      const int k = rank + __popc(mask & ((1u << lane) - 1u));
      if (open && k < got) e[i] = list[k];
      rank += __popc(mask);
    }
  }
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

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
    fork_plan_kernel(const ForkArgs a) {
  __shared__ PlanShared sh;
  cg::this_cluster().sync();   // every CTA has started: its shared memory may be written
  grid_dep_wait();
  grid_dep_launch();
  int first, last, before;
  slice(a.n, &first, &last);
  int mine = 0;
  for (int at = first; at < last; at += kPlanThreads) {
    const int i = at + static_cast<int>(threadIdx.x);
    const int len = i < last ? fork_length(a, i) : 0;
    int total;
    block_rank(len > 0 && len % a.page_size != 0 ? 1 : 0, &total, &sh);
    mine += total;
  }
  const int want = cluster_share(mine, 0, &before, &sh);
  const int got = take_free(a.ref, a.num_pages, want, a.list, 1, &sh);
  for (int at = first; at < last; at += kPlanThreads) {
    const int i = at + static_cast<int>(threadIdx.x);
    const int len = i < last ? fork_length(a, i) : 0;
    const bool need = len > 0 && len % a.page_size != 0;
    int total;
    const int k = before + block_rank(need ? 1 : 0, &total, &sh);
    before += total;
    if (i < last) {
      int f = len < 0 ? kSkip : kNotNeeded;
      if (need) f = k < got ? a.list[k] : kNoPage;
      if (f == kSkip) report(a.status, SMLA_ERR_INDEX_RANGE);
      if (f == kNoPage) report(a.status, SMLA_ERR_POOL_EXHAUSTED);
      a.fresh[i] = f;
    }
  }
}

// Copies `words` 8-byte words from src to dst by the CTA's threads.
__device__ __forceinline__ void copy_rows(uint8_t* pool, int64_t stride, int64_t from, int64_t to,
                                          int rows) {
  const uint8_t* s = pool + from * stride;
  uint8_t* d = pool + to * stride;
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
        if (v >= 0 && v < a.num_pages) atomicAdd(a.ref + v, 1);
      } else if (e == full && rem > 0) {
        v = fresh;
      }
      dst[e] = v;
    }
    if (threadIdx.x == 0) a.kv_lens[c] = len;
  }
  if (rem == 0) return;
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
  int first, last, before;
  slice(a.num_pages, &first, &last);
  const int in_use = count_pages(a.ref, first, last, true, &sh);
  const int used = cluster_share(in_use, 0, &before, &sh);
  // Pages in use below this slice: `before`.  Holes are the free pages below `used`,
  // movers the pages in use at or past it; their ranks follow from `before` alone:
  // free pages below page p = p - (in use below p).
  int below = before;
  for (int at = first; at < last; at += kPlanThreads) {
    const int p = at + static_cast<int>(threadIdx.x);
    const bool u = p < last && __ldcg(a.ref + p) > 0;
    int total;
    const int r = below + block_rank(u ? 1 : 0, &total, &sh);   // pages in use below p
    below += total;
    if (p < last) {
      if (p < used) {
        if (!u) a.holes[p - r] = p;
      } else {
        // a mover's rank is r minus the pages in use below `used`, taken off below
        a.rank_of[p] = u ? r : -1;
      }
    }
  }
  // pages in use below page `used` (the rank of the first mover)
  int low = 0;
  if (used > first && used <= last) {
    int c = 0;
    for (int p = first + threadIdx.x; p < used; p += kPlanThreads) c += __ldcg(a.ref + p) > 0;
    int total;
    block_rank(c, &total, &sh);
    low = before + total;
  }
  int unused;
  const int kept = used > 0 ? cluster_share(low, 1, &unused, &sh) : (cg::this_cluster().sync(), 0);
  const int moved = used - kept;
  // counts: each thread of a move reads and writes both of its pages' counts itself, so
  // ref_out may be ref
  for (int at = first; at < last; at += kPlanThreads) {
    const int p = at + static_cast<int>(threadIdx.x);
    if (p >= last) continue;
    const int c = a.ref[p];
    if (p < used) {
      if (c > 0) a.ref_out[p] = c;
    } else if (c > 0) {
      const int k = a.rank_of[p] - kept;
      a.movers[k] = p;
      a.ref_out[a.holes[k]] = c;
      a.ref_out[p] = 0;
    } else {
      a.ref_out[p] = c;
    }
  }
  const int64_t step = static_cast<int64_t>(kPlanCtas) * kPlanThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x; i < a.entries; i += step) {
    int v = a.table[i];
    if (v >= a.num_pages) {
      report(a.status, SMLA_ERR_INDEX_RANGE);
    } else if (v >= used) {
      const int r = a.rank_of[v];
      if (r >= 0) v = a.holes[r - kept];
      else report(a.status, SMLA_ERR_INDEX_RANGE);
    }
    a.table_out[i] = v;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.info[0] = used;
    a.info[1] = moved;
  }
}

// Moves the listed pages: a CTA takes chunks of kMoveRows rows in turn.
constexpr int kMoveRows = 16;
__global__ void __launch_bounds__(256) compact_move_kernel(const CompactArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int moved = a.info[1];
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
  st = check_workspace(c, workspace, workspace_bytes);
  if (st != SMLA_OK) return st;
  int* status = nullptr;
  st = ready(&status);
  if (st != SMLA_OK) return st;
  char* ws = static_cast<char*>(workspace);
  return done(launch_programmatic(reserve_kernel, dim3(kPlanCtas), dim3(kPlanThreads), 0,
                                  reinterpret_cast<cudaStream_t>(stream), ref_count, block_table,
                                  target_lens, c->num_seqs, c->max_pages, c->page_size, c->num_pages,
                                  reinterpret_cast<int32_t*>(ws),
                                  reinterpret_cast<int32_t*>(ws + 3 * list_bytes(c)), status));
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
