// Selection over beams and vocabulary (smla_beam_select).  Declared and documented in
// include/smla.h.
//
// For row r = group * beams + beam with logits x and score c, a candidate's value is
//     c + (x - M) - ln sum exp(x - M),     M = max x,
// and each group's num_out largest are wanted.  Two launches: segments of 8,192 logits each leave
// their maximum, their sum of exponentials and their own num_out best; a CTA a group joins them.
//
// The logits are read once, into registers.  Best of a segment: the largest logits of 2 num_out (or
// more) parts of it have a num_out-th largest, which at least num_out logits reach and few others
// do, so those go to a list in shared memory that is ranked by counting.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/smla.h"
#include "smla_cache_host.h"
#include "smla_internal.h"
#include "smla_ptx.cuh"

namespace smla {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kEach = 32;                         // logits of a thread
constexpr int kSegment = kThreads * kEach;
constexpr int kMaxOut = 64;
constexpr int kList = 1024;                       // candidates of a segment that are ranked by counting
constexpr unsigned long long kNone = 0;           // no candidate: below every key

struct BeamArgs {
  const void* logits;
  int64_t row_stride;             // elements
  const float* scores;
  const uint8_t* finished;
  int32_t *parents, *tokens;
  float* out_scores;
  // workspace: [row][segment] of maximum and sum, [row][segment][num_out] of keys, descending
  float2* stats;
  unsigned long long* best;
  int beams, vocab, num_out, segments, end_token;
  int* status;
};

__device__ __forceinline__ void report_range(int* status) { atomicCAS(status, 0, SMLA_ERR_RANGE); }

// Larger value first, then the lower token: one number.
__device__ __forceinline__ uint32_t sortable(float x) {
  const uint32_t b = __float_as_uint(x);
  return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unsortable(uint32_t u) { return __uint_as_float((u >> 31) ? u & 0x7fffffffu : ~u); }
__device__ __forceinline__ unsigned long long key_of(float x, int token) {
  x = x == 0.f ? 0.f : x;         // -0 is 0
  return static_cast<unsigned long long>(sortable(x)) << 32 | ~static_cast<uint32_t>(token);
}
__device__ __forceinline__ float key_value(unsigned long long k) { return unsortable(static_cast<uint32_t>(k >> 32)); }
__device__ __forceinline__ int key_token(unsigned long long k) { return static_cast<int>(~static_cast<uint32_t>(k)); }

// The largest key of the warp, in every lane.
__device__ __forceinline__ unsigned long long warp_max(unsigned long long k) {
  const uint32_t hi = static_cast<uint32_t>(k >> 32), top = __reduce_max_sync(0xffffffffu, hi);
  const uint32_t lo = __reduce_max_sync(0xffffffffu, hi == top ? static_cast<uint32_t>(k) : 0u);
  return static_cast<unsigned long long>(top) << 32 | lo;
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// e^d for d <= 0: log2(e) in two parts, since the first alone is off by 1.3e-8 and every term of a sum
// by 1e-7 in the same direction.
__device__ __forceinline__ float exp_of(float d) { return exp2_fast(fmaf(d, 1.44269502162933349609f, d * 1.92596299e-8f)); }

// Words of 16, 4 or 2 bytes.
template <int BYTES>
struct Word;
template <>
struct Word<16> { using type = uint4; };
template <>
struct Word<4> { using type = unsigned int; };
template <>
struct Word<2> { using type = unsigned short; };

// BYTES: of a load, what the start of every row is aligned to.  Which thread adds which logits goes by
// their place in the row alone, so that equal rows have equal sums, and ties are ties.
template <class T, int BYTES>
__global__ void __launch_bounds__(kThreads) segment_kernel(const BeamArgs a) {
  constexpr int kPer = BYTES / sizeof(T), kVecs = kEach / kPer;       // logits of a word; words a thread
  __shared__ float part[2 * kMaxOut], warp_top[kWarps], warp_sum[kWarps];
  __shared__ float least;
  __shared__ int count;
  __shared__ unsigned long long list[kList];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int seg = blockIdx.x, row = blockIdx.y;
  grid_dep_wait();
  grid_dep_launch();
  if (a.finished != nullptr && a.finished[row] != 0) return;
  if (tid == 0) {
    count = 0;
    least = INFINITY;
  }
  const T* base = static_cast<const T*>(a.logits) + row * a.row_stride;
  const int first = seg * kSegment + tid * kPer;            // of word 0
  float x[kEach];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int at = first + j * kThreads * kPer;
    if (at + kPer <= a.vocab) {
      const auto w = __ldcs(reinterpret_cast<const typename Word<BYTES>::type*>(base + at));
      const T* v = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int e = 0; e < kPer; ++e) x[j * kPer + e] = to_float(v[e]);
    } else {
#pragma unroll
      for (int e = 0; e < kPer; ++e) x[j * kPer + e] = at + e < a.vocab ? to_float(base[at + e]) : -INFINITY;
    }
  }
  auto token = [&](int i) { return first + (i / kPer) * kThreads * kPer + i % kPer; };
  float mine = x[0];
#pragma unroll
  for (int i = 1; i < kEach; ++i) mine = fmaxf(mine, x[i]);
  // maxima of the parts: 16, 32, 64 or 128 of them
  const int lanes = a.num_out <= 8 ? 16 : a.num_out <= 16 ? 8 : a.num_out <= 32 ? 4 : 2, parts = kThreads / lanes;
  float top = mine;
  for (int o = 1; o < 32; o <<= 1) {
    if (o == lanes && lane % lanes == 0) part[tid / lanes] = top;
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  if (lane == 0) warp_top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, warp_top[w]);
  if (tid < parts) {
    const float p = part[tid];
    int rank = 0;
    for (int j = 0; j < parts; ++j) rank += part[j] > p || (part[j] == p && j < tid);
    if (rank == a.num_out - 1) least = fmaxf(p, -3.402823466e38f);   // -infinity is no candidate
  }
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  if (top == -INFINITY) {        // nothing but -infinity, or NaN, which a maximum drops
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (x[i] != x[i]) sum[0] = x[i];
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i) sum[i % 4] += exp_of(x[i] - top);
  }
  float s = (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) warp_sum[warp] = s;
  __syncthreads();
  if (mine >= least) {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (x[i] >= least) {
        const int at = atomicAdd(&count, 1);
        if (at < kList) list[at] = key_of(x[i], token(i));
      }
  }
  const int64_t slot = static_cast<int64_t>(row) * a.segments + seg;
  if (tid == 0) {
    float all = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) all += warp_sum[w];
    a.stats[slot] = make_float2(top, all);        // a NaN or +infinity leaves a sum that is not finite
  }
  __syncthreads();
  unsigned long long* out = a.best + slot * a.num_out;
  const int n = count;
  if (n <= kList) {
    for (int i = tid; i < n; i += kThreads) {
      const unsigned long long k = list[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += list[j] > k;
      if (rank < a.num_out) out[rank] = k;
    }
    for (int i = n + tid; i < a.num_out; i += kThreads) out[i] = kNone;
    return;
  }
  // more equal logits than the list holds: one after the other, each the largest below the last
  unsigned long long last = ~0ull;
  for (int i = 0; i < a.num_out; ++i) {
    unsigned long long k = kNone;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const unsigned long long c = x[j] >= least ? key_of(x[j], token(j)) : kNone;
      if (c < last && c > k) k = c;
    }
    k = warp_max(k);
    __syncthreads();
    if (lane == 0) list[warp] = k;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) k = list[w] > k ? list[w] : k;
    if (tid == 0) out[i] = k;
    last = k;
  }
}

// ln x for x >= 1, in 64 bits where 32 would round the whole: the power of two apart, the rest in
// 32 bits (3e-8).
__device__ __forceinline__ double log_of(float x) {
  int e = static_cast<int>(__float_as_uint(x) >> 23) - 127;
  float m = __uint_as_float((__float_as_uint(x) & 0x007fffffu) | 0x3f800000u);
  if (m > 1.4142135f) {
    m *= 0.5f;
    ++e;
  }
  return e * 0.693147180559945309417 + static_cast<double>(log1pf(m - 1.f));
}
__device__ __forceinline__ unsigned long long sortable64(double x) {
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(x));
  return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}

constexpr int kHeld = 16;          // keys of a lane while a beam's lists are joined

// A CTA a group.  A warp joins the segments of a beam, beam after beam; then one warp takes the
// group's best, one at a time, from the heads of the beams' lists.
__global__ void __launch_bounds__(kThreads) join_kernel(const BeamArgs a) {
  extern __shared__ unsigned long long lists[];          // [beams][num_out] keys
  __shared__ double base[kMaxOut], shift[kMaxOut], log_sum[kMaxOut];       // of a beam: score, M, ln sum
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = blockIdx.x, n = a.num_out;
  grid_dep_wait();
  grid_dep_launch();
  for (int b = warp; b < a.beams; b += kWarps) {
    const int row = group * a.beams + b;
    const float score = a.scores[row];
    unsigned long long* mine = lists + b * n;
    if (a.finished != nullptr && a.finished[row] != 0) {
      const bool fine = fabsf(score) < INFINITY;
      for (int i = lane; i < n; i += 32) mine[i] = i == 0 && fine ? key_of(0.f, a.end_token) : kNone;
      if (lane == 0) {
        base[b] = score;
        shift[b] = log_sum[b] = 0.0;
        if (!fine && score != -INFINITY) report_range(a.status);
      }
      continue;
    }
    const float2* stats = a.stats + static_cast<int64_t>(row) * a.segments;
    float top = -INFINITY;
    bool bad = false;
    for (int s = lane; s < a.segments; s += 32) {
      const float2 t = stats[s];
      top = fmaxf(top, t.x);
      bad |= !(t.y < INFINITY);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float sum = 0.f;
    for (int s = lane; s < a.segments; s += 32) {
      const float2 t = stats[s];
      if (t.y > 0.f) sum = fmaf(t.y, exp_of(t.x - top), sum);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    bad = __any_sync(0xffffffffu, bad) || (!(fabsf(score) < INFINITY) && score != -INFINITY);
    if (bad && lane == 0) report_range(a.status);
    const bool empty = bad || top == -INFINITY || score == -INFINITY;
    if (lane == 0) {
      base[b] = score;
      shift[b] = top;
      log_sum[b] = empty ? 0.0 : log_of(sum);
    }
    // the n largest of segments * n keys: the best so far and the next ones, kHeld a lane at a time
    const unsigned long long* best = a.best + static_cast<int64_t>(row) * a.segments * n;
    const int64_t total = empty ? 0 : static_cast<int64_t>(a.segments) * n;
    for (int i = lane; i < n; i += 32) mine[i] = kNone;
    __syncwarp();
    for (int64_t at = 0; at < total; at += 32 * (kHeld - 2)) {
      unsigned long long held[kHeld];
#pragma unroll
      for (int i = 0; i < kHeld - 2; ++i) {
        const int64_t j = at + i * 32 + lane;
        held[i] = j < total ? best[j] : kNone;
      }
      held[kHeld - 2] = lane < n ? mine[lane] : kNone;
      held[kHeld - 1] = lane + 32 < n ? mine[lane + 32] : kNone;
      __syncwarp();
      for (int i = 0; i < n; ++i) {
        unsigned long long k = held[0];
#pragma unroll
        for (int j = 1; j < kHeld; ++j) k = held[j] > k ? held[j] : k;
        k = warp_max(k);
#pragma unroll
        for (int j = 0; j < kHeld; ++j) held[j] = held[j] == k ? kNone : held[j];
        if (lane == 0) mine[i] = k;
      }
      __syncwarp();
    }
  }
  __syncthreads();
  if (warp != 0) return;
  // x - M first: logits of any size keep their differences; the logarithm last: what is equal but for
  // rounding in beams of equal sums stays equal
  auto value = [&](int b, unsigned long long k) {
    return (base[b] + (static_cast<double>(key_value(k)) - shift[b])) - log_sum[b];
  };
  // the heads of beams lane and lane + 32
  int at[2] = {0, 0};
  auto head = [&](int i) {
    const int b = lane + 32 * i;
    const unsigned long long k = b < a.beams && at[i] < n ? lists[b * n + at[i]] : kNone;
    return k == kNone ? 0ull : sortable64(value(b, k));
  };
  unsigned long long h[2] = {head(0), head(1)};
  for (int i = 0; i < n; ++i) {
    const int own = h[1] > h[0] ? 1 : 0;              // equal: the lower beam
    const unsigned long long v = own ? h[1] : h[0], k = warp_max(v);
    const int beam = static_cast<int>(__reduce_min_sync(0xffffffffu, v == k ? lane + 32 * own : 0x7fffffffu));
    const int64_t o = static_cast<int64_t>(group) * n + i;
    if (k == 0) {
      if (lane == 0) {
        a.parents[o] = a.tokens[o] = -1;
        a.out_scores[o] = -INFINITY;
      }
      continue;
    }
    if (beam % 32 == lane) {
      const int w = beam / 32;
      const unsigned long long c = lists[beam * n + at[w]];
      a.parents[o] = group * a.beams + beam;
      a.tokens[o] = key_token(c);
      a.out_scores[o] = static_cast<float>(value(beam, c));
      ++at[w];
      h[w] = head(w);
    }
    __syncwarp();
  }
}

int check_beam(const smla_beam_params* p) {
  if (p == nullptr || p->reserved != 0) return SMLA_ERR_INVALID_ARG;
  if (p->groups < 1 || p->beams < 1 || p->vocab < 1 || p->num_out < 1 || p->row_stride < p->vocab) return SMLA_ERR_INVALID_ARG;
  if (p->logits_type != SMLA_FLOAT32 && p->logits_type != SMLA_BFLOAT16 && p->logits_type != SMLA_FLOAT16)
    return SMLA_ERR_INVALID_ARG;
  if (p->beams > kMaxOut || p->num_out > kMaxOut || p->vocab > (1 << 24) ||
      static_cast<int64_t>(p->groups) * p->beams > 65535 || p->row_stride > (int64_t{1} << 40))
    return SMLA_ERR_UNSUPPORTED_SHAPE;
  return SMLA_OK;
}
int segments_of(const smla_beam_params* p) { return (p->vocab - 1) / kSegment + 1; }

// The widest load that every row's start allows.
template <class T>
auto segment_of(const void* logits, int64_t row_stride) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(logits) | static_cast<uintptr_t>(row_stride) * sizeof(T);
  if (at % 16 == 0) return segment_kernel<T, 16>;
  if constexpr (sizeof(T) == 2) {
    if (at % 4 != 0) return segment_kernel<T, 2>;
  }
  return segment_kernel<T, 4>;
}

size_t lay_out(const smla_beam_params* p, char* base, BeamArgs* a) {
  const size_t slots = static_cast<size_t>(p->groups) * p->beams * segments_of(p);
  a->stats = reinterpret_cast<float2*>(base);
  const size_t at = round256(slots * sizeof(float2));
  a->best = reinterpret_cast<unsigned long long*>(base + at);
  return at + round256(slots * p->num_out * sizeof(unsigned long long));
}

}  // namespace
}  // namespace smla

using namespace smla;   // NOLINT: the entry points below are this file's own

extern "C" {

int smla_beam_workspace_size(const smla_beam_params* p, size_t* bytes) {
  const int st = check_beam(p);
  if (st != SMLA_OK) return st;
  if (bytes == nullptr) return SMLA_ERR_INVALID_ARG;
  BeamArgs a;
  *bytes = lay_out(p, nullptr, &a);
  return SMLA_OK;
}

int smla_beam_select(const void* logits, const float* scores, const uint8_t* finished, int32_t* parents,
                     int32_t* tokens, float* out_scores, const smla_beam_params* p, void* workspace,
                     size_t workspace_bytes, smla_stream_t stream) {
  int st = check_beam(p);
  if (st != SMLA_OK) return st;
  if (finished != nullptr && (p->end_token < 0 || p->end_token >= p->vocab)) return SMLA_ERR_INVALID_ARG;
  const uintptr_t size = p->logits_type == SMLA_FLOAT32 ? 4 : 2;
  if (logits == nullptr || !aligned(logits, size) || scores == nullptr || !aligned(scores, 4) || !ints_ok(parents) ||
      !ints_ok(tokens) || out_scores == nullptr || !aligned(out_scores, 4) || workspace == nullptr || !aligned(workspace, 256))
    return SMLA_ERR_INVALID_ARG;
  BeamArgs a = {logits, p->row_stride, scores, finished, parents, tokens, out_scores, nullptr, nullptr,
                p->beams, p->vocab, p->num_out, segments_of(p), p->end_token, nullptr};
  if (workspace_bytes < lay_out(p, static_cast<char*>(workspace), &a)) return SMLA_ERR_WORKSPACE_TOO_SMALL;
  st = ready(&a.status);
  if (st != SMLA_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid(a.segments, p->groups * p->beams);
  const auto segment = p->logits_type == SMLA_FLOAT32    ? segment_of<float>(logits, p->row_stride)
                       : p->logits_type == SMLA_BFLOAT16 ? segment_of<__nv_bfloat16>(logits, p->row_stride)
                                                         : segment_of<__half>(logits, p->row_stride);
  st = done(launch_programmatic(segment, grid, dim3(kThreads), 0, s, a));
  if (st != SMLA_OK) return st;
  const size_t lists = sizeof(unsigned long long) * p->beams * p->num_out;      // 32 KB at most
  return done(launch_programmatic(join_kernel, dim3(p->groups), dim3(kThreads), lists, s, a));
}

}  // extern "C"
