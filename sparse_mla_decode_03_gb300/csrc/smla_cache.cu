// The pages of the paged cache (smla_cache_reserve, _fork, _free, _compact).  Declared and
// documented in include/smla.h.
//
// Page calls.  A page is free exactly when its count is 0, so no free list is kept: a
// call scans the counts.  The scans and the rankings that depend on one another run as
// one thread-block cluster of 8 CTAs (hardware cluster barriers between the phases, a
// CTA's slice of the pages or table each), so a call is one launch, plus one wide launch
// where rows of the cache move.  Page calls are bound by launches and by the trips to memory
// and cluster barriers of a plan: free 4 us, fork 10 + 5.5 (512 children 11 + 8), reserve 6 (of
// 528 rows and 32,768 pages 12.5), compaction's plan 7.5 (32,768 pages 11).
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/smla.h"
#include "smla_cache_host.h"
#include "smla_cache_plan.cuh"
#include "smla_cache_rows.cuh"
#include "smla_internal.h"
#include "smla_ptx.cuh"

namespace smla {
namespace {

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
    each_entry(a.max_pages, [&](int e) {
      int v = -1;
      if (e < full) {
        v = src[e];
      } else if (e == full && rem > 0) {
        v = fresh >= 0 ? fresh : src[e];
      }
      if (v >= a.num_pages) report(a.status, SMLA_ERR_INDEX_RANGE);
      else if (v >= 0 && e < full) atomicAdd(a.ref + v, 1);
      dst[e] = v;
    });
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
  each_entry(max_pages, [&](int i) {
    if (e[i] < 0) return;
    const int p = atomicExch(e + i, -1);   // a row listed twice gives its pages back once
    if (p < 0) return;
    if (p >= num_pages) {
      report(status, SMLA_ERR_INDEX_RANGE);
    } else if (atomicSub(ref + p, 1) <= 0) {
      atomicAdd(ref + p, 1);
      report(status, SMLA_ERR_INDEX_RANGE);
    }
  });
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

}  // namespace
}  // namespace smla

using namespace smla;   // NOLINT: the entry points below are this file's own

extern "C" {

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
  if (!pool_ok(kv_pages, c) || !ints_ok(ref_count) || !ints_ok(block_table) || !ints_ok(kv_lens))
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
  if (!pool_ok(kv_pages, c) || !ints_ok(ref_count) || !ints_ok(block_table) || !ints_ok(ref_count_out) ||
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
