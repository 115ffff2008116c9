// Reordering of the paged cache by parents (smla_cache_reorder): row r of the table goes on from
// the row that parents[r] names, in place.  Declared and documented in include/smla.h.
//
// Two launches.  The first cluster of the plan finds the child that takes each row over (the lowest),
// gives the pages of rows without a child back, and only then ranks the free pages for the last pages
// that further children copy, so a beam that is dropped makes room for the one that is doubled.  Its other
// clusters meanwhile copy the table and the lengths aside, since the second launch overwrites the rows
// that others still read.
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

struct ReorderArgs {
  uint8_t* pool;
  int32_t *ref, *table, *kv_lens;
  const int32_t* parents;
  int32_t *old_table, *old_lens;      // workspace, as are the lists
  int32_t *first, *list, *fresh;      // lowest child of each row; free pages taken; the new page of each child
  int rows, max_pages, page_size, num_pages;
  int64_t stride;
  int* status;
};
constexpr int kNobody = 0x7fffffff;
constexpr int kNoPage = -1, kNotNeeded = -2;

// The length of row p that its further children see: within the table.
__device__ __forceinline__ int parent_length(const ReorderArgs& a, const int32_t* lens, int p) {
  const int64_t most = static_cast<int64_t>(a.max_pages) * a.page_size;
  const int len = lens[p];
  return len < 0 ? 0 : static_cast<int>(min(static_cast<int64_t>(len), most));
}
__device__ __forceinline__ int parent_of(const ReorderArgs& a, int r) {
  const int p = __ldg(a.parents + r);
  return p < a.rows ? p : -1;
}
// Whether child r, which does not take row p over, copies a last page that is partly filled and mapped.
__device__ __forceinline__ bool takes_page(const ReorderArgs& a, int p) {
  const int len = parent_length(a, a.kv_lens, p);
  if (len % a.page_size == 0) return false;
  const int page = a.table[static_cast<int64_t>(p) * a.max_pages + len / a.page_size];
  return page >= 0 && page < a.num_pages;
}

// Exclusive sums of two counts over the CTA's threads; *total gets the sums.  All threads call.
__device__ __forceinline__ int2 block_rank2(int2 v, int2* total, int2* warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int2 s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, s.x, o), y = __shfl_up_sync(0xffffffffu, s.y, o);
    if (lane >= o) {
      s.x += x;
      s.y += y;
    }
  }
  if (lane == 31) warps[warp] = s;
  __syncthreads();
  int2 w = warps[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, w.x, o), y = __shfl_up_sync(0xffffffffu, w.y, o);
    if (lane >= o) {
      w.x += x;
      w.y += y;
    }
  }
  *total = make_int2(__shfl_sync(0xffffffffu, w.x, 31), __shfl_sync(0xffffffffu, w.y, 31));
  const int from = warp > 0 ? warp - 1 : 0;
  const int bx = __shfl_sync(0xffffffffu, w.x, from), by = __shfl_sync(0xffffffffu, w.y, from);
  return make_int2(s.x - v.x + (warp > 0 ? bx : 0), s.y - v.y + (warp > 0 ? by : 0));
}

// Rows whose lowest children every CTA of the plan finds for itself, in shared memory; more: together, in the
// workspace, which takes two cluster barriers.
constexpr int kOwnRows = 8192;
constexpr int kGive = 128;

// Bound by latency: a launch, four trips to memory one after the other (parents, lengths, table; counts) and three
// cluster barriers: 8.5 us for 8 rows and 8,192 pages (10.8 when a warp gave a row's pages back 32 at a time), 11 for
// 512 rows and 32,768 (19 when the lowest children went through the workspace there too).
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
    reorder_plan_kernel(const ReorderArgs a) {
  __shared__ PlanShared sh;
  __shared__ int2 warps[32];
  __shared__ int own[kOwnRows];
  cg::this_cluster().sync();   // every CTA has started: its shared memory may be written
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x >= kPlanCtas) {
    const int64_t entries = static_cast<int64_t>(a.rows) * a.max_pages;
    const int64_t step = static_cast<int64_t>(gridDim.x - kPlanCtas) * kPlanThreads;
    const int64_t i0 = static_cast<int64_t>(blockIdx.x - kPlanCtas) * kPlanThreads + threadIdx.x;
    for (int64_t i = i0; i < entries; i += step) a.old_table[i] = a.table[i];
    for (int64_t i = i0; i < a.rows; i += step) a.old_lens[i] = a.kv_lens[i];
    return;
  }
  const bool few = a.rows <= kOwnRows;
  const int tid = static_cast<int>(threadIdx.x), cta = static_cast<int>(blockIdx.x);
  constexpr int kAll = kPlanCtas * kPlanThreads;
  {
    int* first = few ? own : a.first;
    const int r0 = few ? tid : cta * kPlanThreads + tid, step = few ? kPlanThreads : kAll;
    for (int r = r0; r < a.rows; r += step) first[r] = kNobody;
    if (few) __syncthreads();
    else cg::this_cluster().sync();
    for (int r = r0; r < a.rows; r += step) {
      const int p = __ldg(a.parents + r);
      if (p >= a.rows) report(a.status, SMLA_ERR_INDEX_RANGE);
      else if (p >= 0) atomicMin(first + p, r);
    }
    if (few) __syncthreads();
    else cg::this_cluster().sync();
  }
  auto first_of = [&](int p) { return few ? own[p] : __ldcg(a.first + p); };
  // this CTA's rows, each thread a run of them: who copies a page
  const int per = (a.rows + kPlanCtas - 1) / kPlanCtas, row0 = min(a.rows, cta * per), row1 = min(a.rows, row0 + per);
  const int run = (row1 - row0 + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(row1, row0 + tid * run), r1 = min(row1, r0 + run);
  auto copies = [&](int r) {
    const int p = parent_of(a, r);
    return p >= 0 && first_of(p) != r && takes_page(a, p);
  };
  uint32_t who = 0;               // run <= 8: 65,535 rows on 8,192 threads
  for (int r = r0; r < r1; ++r) {
    if (few) a.first[r] = own[r];         // for the next launch
    who |= copies(r) ? 1u << (r - r0) : 0u;
  }
  // rows that nobody goes on from give their pages back: a warp takes kGive entries of one, all on their way at once
  const int lane = tid & 31, pieces = (a.max_pages - 1) / kGive + 1;
  const int64_t units = static_cast<int64_t>(a.rows) * pieces;
  for (int64_t u = (cta * kPlanThreads + tid) / 32; u < units; u += kAll / 32) {
    const int r = static_cast<int>(u / pieces), e0 = static_cast<int>(u - static_cast<int64_t>(r) * pieces) * kGive + lane;
    if (first_of(r) != kNobody) continue;
    const int32_t* e = a.table + static_cast<int64_t>(r) * a.max_pages;
    int page[kGive / 32], count[kGive / 32];
#pragma unroll
    for (int k = 0; k < kGive / 32; ++k) page[k] = e0 + 32 * k < a.max_pages ? e[e0 + 32 * k] : -1;
#pragma unroll
    for (int k = 0; k < kGive / 32; ++k) {
      count[k] = 1;
      if (page[k] >= 0 && page[k] < a.num_pages) count[k] = atomicSub(a.ref + page[k], 1);
    }
#pragma unroll
    for (int k = 0; k < kGive / 32; ++k) {
      if (count[k] <= 0) atomicAdd(a.ref + page[k], 1);
      if (count[k] <= 0 || page[k] >= a.num_pages) report(a.status, SMLA_ERR_INDEX_RANGE);
    }
  }
  cg::this_cluster().sync();
  const Part pp = part_of(a.num_pages);
  int2 total, low;
  const int2 rank = block_rank2(make_int2(__popc(who), count_free(a.ref, pp)), &total, warps);
  const int2 all = cluster_share(total, 0, &low, &sh);
  const int got = min(all.x, all.y);
  take_free(a.ref, pp, low.y + rank.y, got, a.list);
  cg::this_cluster().sync();
  int k = low.x + rank.x;
  for (int r = r0; r < r1; ++r) {
    int f = kNotNeeded;
    if ((who >> (r - r0)) & 1) {
      f = k < got ? __ldcg(a.list + k) : kNoPage;
      ++k;
      if (f == kNoPage) report(a.status, SMLA_ERR_POOL_EXHAUSTED);
    }
    a.fresh[r] = f;
  }
}

constexpr int kCopyRows = 16;   // rows of a partial page that one CTA copies

// Grid (rows, row groups of a page): group 0 also writes the row of the table.  A launch, two trips to memory and the
// copies: 4.6 us for 8 rows, 7 for 512 of which half copy 56 rows.
__global__ void __launch_bounds__(256) reorder_apply_kernel(const ReorderArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int r = blockIdx.x, p = parent_of(a, r);
  int32_t* dst = a.table + static_cast<int64_t>(r) * a.max_pages;
  const int fresh = a.fresh[r];
  if (p < 0 || fresh == kNoPage) {
    if (blockIdx.y != 0) return;
    each_entry(a.max_pages, [&](int e) { dst[e] = -1; });
    if (threadIdx.x == 0) a.kv_lens[r] = 0;
    return;
  }
  const int32_t* src = a.old_table + static_cast<int64_t>(p) * a.max_pages;
  if (a.first[p] == r) {        // takes the row over as it is
    if (p == r || blockIdx.y != 0) return;
    each_entry(a.max_pages, [&](int e) { dst[e] = src[e]; });
    if (threadIdx.x == 0) a.kv_lens[r] = a.old_lens[p];
    return;
  }
  const int len = parent_length(a, a.old_lens, p), full = len / a.page_size, rem = len % a.page_size;
  if (blockIdx.y == 0) {
    each_entry(a.max_pages, [&](int e) {
      int v = -1;
      if (e < full) v = src[e];
      else if (e == full && rem > 0) v = fresh >= 0 ? fresh : src[e];
      if (v >= a.num_pages) report(a.status, SMLA_ERR_INDEX_RANGE);
      else if (v >= 0 && e < full) atomicAdd(a.ref + v, 1);
      dst[e] = v;
    });
    if (threadIdx.x == 0) {
      a.kv_lens[r] = len;
      if (a.old_lens[p] != len) report(a.status, SMLA_ERR_INDEX_RANGE);
    }
  }
  if (fresh < 0) return;
  const int64_t from = static_cast<int64_t>(src[full]) * a.page_size, to = static_cast<int64_t>(fresh) * a.page_size;
  for (int r0 = blockIdx.y * kCopyRows; r0 < rem; r0 += gridDim.y * kCopyRows)
    copy_rows(a.pool, a.stride, from + r0, to + r0, min(kCopyRows, rem - r0));
}

// The workspace; base may be null to size it.
size_t lay_out(const smla_cache_params* c, char* base, ReorderArgs* a) {
  size_t at = 0;
  auto take = [&](size_t ints) {
    int32_t* p = reinterpret_cast<int32_t*>(base + at);
    at += round256(4 * ints);
    return p;
  };
  const size_t rows = static_cast<size_t>(c->num_seqs);
  a->first = take(rows);
  a->list = take(rows);
  a->fresh = take(rows);
  a->old_lens = take(rows);
  a->old_table = take(rows * c->max_pages);
  return at;
}

}  // namespace
}  // namespace smla

using namespace smla;   // NOLINT: the entry points below are this file's own

extern "C" {

int smla_cache_reorder_workspace_size(const smla_cache_params* c, size_t* bytes) {
  const int st = check_cache(c);
  if (st != SMLA_OK) return st;
  if (bytes == nullptr) return SMLA_ERR_INVALID_ARG;
  ReorderArgs a;
  *bytes = lay_out(c, nullptr, &a);
  return SMLA_OK;
}

int smla_cache_reorder(void* kv_pages, int32_t* ref_count, int32_t* block_table, int32_t* kv_lens,
                       const int32_t* parents, const smla_cache_params* c, void* workspace,
                       size_t workspace_bytes, smla_stream_t stream) {
  int st = check_cache(c);
  if (st != SMLA_OK) return st;
  if (!pool_ok(kv_pages, c) || !ints_ok(ref_count) || !ints_ok(block_table) || !ints_ok(kv_lens) || !ints_ok(parents))
    return SMLA_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256)) return SMLA_ERR_INVALID_ARG;
  ReorderArgs a = {static_cast<uint8_t*>(kv_pages), ref_count, block_table, kv_lens, parents, nullptr, nullptr,
                   nullptr, nullptr, nullptr, c->num_seqs, c->max_pages, c->page_size, c->num_pages,
                   c->kv_row_stride, nullptr};
  if (workspace_bytes < lay_out(c, static_cast<char*>(workspace), &a)) return SMLA_ERR_WORKSPACE_TOO_SMALL;
  st = ready(&a.status);
  if (st != SMLA_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // clusters that copy the table aside: eight entries a thread
  const int64_t entries = static_cast<int64_t>(c->num_seqs) * c->max_pages;
  const int64_t copies = (entries - 1) / (8 * kPlanCtas * kPlanThreads) + 1;
  const unsigned clusters = 1 + static_cast<unsigned>(copies < 18 ? copies : 18);
  st = done(launch_programmatic(reorder_plan_kernel, dim3(clusters * kPlanCtas), dim3(kPlanThreads), 0, s, a));
  if (st != SMLA_OK) return st;
  const int groups = (c->page_size - 1) / kCopyRows + 1;
  return done(launch_programmatic(reorder_apply_kernel, dim3(c->num_seqs, groups < 64 ? groups : 64), dim3(256), 0, s, a));
}

}  // extern "C"
