// Selection over beams and vocabulary (smla_beam_select).  Declared and documented in
// include/smla.h.
//
// For row r = group * beams + beam with logits x and score c, a candidate's value is
//     c + (x - M) - ln sum exp(x - M),     M = max x,
// and each group's num_out largest are wanted.  Two launches.  The first reads the logits once: warps
// go over runs of them, 2 KB (a step) at a time, and leave each step's maximum and each run's sum of
// exponentials; they meet nobody and keep no candidates.  The second, a CTA a group, finds a border from
// the maxima that at least num_out candidates reach and few steps do (bit by bit, a count of the CTA's
// threads a bit), reads those few steps again, and ranks what reaches the border by counting.  Where too many
// steps reach it (wide groups, of which few beams lead), the border comes from the steps' maxima themselves; where
// too many logits do (few steps, beams far apart), from those steps' logits; and where too many are equal, the
// steps that may hold something better are gone through one by one.
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

constexpr int kThreads = 512;                     // of the CTA that joins a group
constexpr int kWarps = kThreads / 32;
constexpr int kRunWarps = 4;                      // of a CTA that goes over runs
constexpr int kRegs = 16;                         // registers of a lane's logits
template <class T>
constexpr int kEach = 4 * kRegs / static_cast<int>(sizeof(T));        // logits of a lane: 16 or 32
template <class T>
constexpr int kStep = 32 * kEach<T>;              // of a warp
constexpr int kMaxOut = 64;
constexpr int kList = 512;                        // candidates that are ranked by counting
constexpr int kBlocks = 512;                      // steps that are read again

struct BeamArgs {
  const void* logits;
  int64_t row_stride;             // elements
  const float* scores;
  const uint8_t* finished;
  int32_t *parents, *tokens;
  float* out_scores;
  // workspace: [row][run] of maximum and sum, [row][step] of maximum
  float2* stats;
  float* maxima;
  int rows, beams, vocab, num_out, steps, runs, end_token;      // steps of a row, and its runs
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

// The largest t >= t0 of which count(t) (the same in all threads, falling in t) is `least` at least, from bit `bit`
// on, above which it is t0; any of which it is `most` at most will do.
template <class F>
__device__ __forceinline__ uint32_t border_of(uint32_t t, uint32_t bit, int least, int most, F count) {
  for (; bit != 0; bit >>= 1) {
    const int c = count(t | bit);
    if (c >= least) {
      t |= bit;
      if (c <= most) break;
    }
  }
  return t;
}

// Words of 16, 4 or 2 bytes.
template <int BYTES>
struct Word;
template <>
struct Word<16> { using type = uint4; };
template <>
struct Word<4> { using type = unsigned int; };
template <>
struct Word<2> { using type = unsigned short; };

// A thread's logits as they lie in memory, two of 16 bits to a register, and the maxima of its quarters.
template <class T>
struct Held;
template <>
struct Held<float> {
  static constexpr uint32_t kNothing = 0xff800000u;      // -infinity
  uint32_t w[kRegs];
  __device__ __forceinline__ float at(int i) const { return __uint_as_float(w[i]); }
  __device__ __forceinline__ float top(int quarter) const {
    float m = at(quarter * kRegs / 4);
#pragma unroll
    for (int i = 1; i < kRegs / 4; ++i) m = fmaxf(m, at(quarter * kRegs / 4 + i));
    return m;
  }
};
template <class T>
struct Held16 {
  uint32_t w[kRegs];
  __device__ __forceinline__ float at(int i) const { return i % 2 ? T::high(w[i / 2]) : T::low(w[i / 2]); }
  __device__ __forceinline__ float top(int quarter) const {
    uint32_t m = w[quarter * kRegs / 4];
#pragma unroll
    for (int i = 1; i < kRegs / 4; ++i) m = T::max(m, w[quarter * kRegs / 4 + i]);
    return fmaxf(T::low(m), T::high(m));
  }
};
struct Bf16 {
  static __device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};
struct Fp16 {
  static __device__ __forceinline__ float low(uint32_t w) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(w)));
  }
  static __device__ __forceinline__ float high(uint32_t w) { return low(w >> 16); }
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};
template <>
struct Held<__nv_bfloat16> : Held16<Bf16> {
  static constexpr uint32_t kNothing = 0xff80u;
};
template <>
struct Held<__half> : Held16<Fp16> {
  static constexpr uint32_t kNothing = 0xfc00u;
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

// log2(e) in two parts, since the first alone is off by 1.3e-8 and every term of a sum by 1e-7 in the same
// direction.
constexpr float kLog2e0 = 1.44269502162933349609f, kLog2e1 = 1.92596299e-8f;
// e^d for two d <= 0
__device__ __forceinline__ Two exp_of(Two d) {
  float x, y;
  fma2(d, Two(kLog2e0), d * Two(kLog2e1)).get(&x, &y);
  return Two(exp2_fast(x), exp2_fast(y));
}

// The row's last logits, element by element; out of line, once a row.
template <class T>
__device__ __noinline__ uint4 load_last(const T* base, int at, int vocab) {
  uint32_t v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (sizeof(T) == 4) {
      v[k] = at + k < vocab ? reinterpret_cast<const uint32_t*>(base)[at + k] : Held<T>::kNothing;
    } else {
      const unsigned short* half = reinterpret_cast<const unsigned short*>(base);
      const uint32_t lo = at + 2 * k < vocab ? half[at + 2 * k] : Held<T>::kNothing;
      const uint32_t hi = at + 2 * k + 1 < vocab ? half[at + 2 * k + 1] : Held<T>::kNothing;
      v[k] = lo | hi << 16;
    }
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

template <class T, int BYTES>
__device__ __forceinline__ void load_step(const T* base, int first, int vocab, Held<T>& x) {
  constexpr int kPer = BYTES / sizeof(T), kWords = kEach<T> / kPer;       // logits of a word; words a lane
#pragma unroll
  for (int j = 0; j < kWords; ++j) {
    const int at = first + j * 32 * kPer;
    const bool whole = at + kPer <= vocab;
    const auto* from = reinterpret_cast<const typename Word<BYTES>::type*>(base + at);
    constexpr uint32_t kNothing = Held<T>::kNothing, kTwo = sizeof(T) == 4 ? kNothing : kNothing * 0x10001u;
    if constexpr (BYTES == 16) {
      uint4 w = make_uint4(kTwo, kTwo, kTwo, kTwo);
      if (whole) w = __ldcs(from);
      else if (at < vocab) w = load_last(base, at, vocab);
      x.w[4 * j] = w.x;
      x.w[4 * j + 1] = w.y;
      x.w[4 * j + 2] = w.z;
      x.w[4 * j + 3] = w.w;
    } else if constexpr (BYTES == 4) {
      uint32_t w = kTwo;
      if (whole) w = __ldcs(from);
      else if (at < vocab) w = load_last(base, at, vocab).x;       // the first of two
      x.w[j] = w;
    } else {
      const uint32_t w = whole ? __ldcs(from) : static_cast<unsigned short>(kNothing);
      if (j % 2 == 0) x.w[j / 2] = w;
      else x.w[j / 2] |= w << 16;
    }
  }
}

// BYTES: of a load, what the start of every row is aligned to.  Which lane adds which logits goes by
// their place in the row alone, so that equal rows have equal sums, and ties are ties.
// Bound by memory: 2 KB a warp is on its way, 56 KB an SM (28 warps of 64 at work).  Nine tenths of 512 rows of 131,072
// bf16 logits (the others have ended; 121 MB): 24.8 us, 4.9 TB/s, with the start (issue slots 60 %, exponentials 31 % of
// their pipe).  256 rows: 25.5 us with both launches at 16 bytes a load, 29.9 at 4 and 34.1 at 2 (replayed graphs).
template <class T, int BYTES>
__global__ void __launch_bounds__(kRunWarps * 32, 8) run_kernel(const BeamArgs a) {
  constexpr int kPer = BYTES / sizeof(T);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_wait();
  grid_dep_launch();
  const int64_t slot = static_cast<int64_t>(blockIdx.x) * kRunWarps + warp;
  const int row = static_cast<int>(slot / a.runs), run = static_cast<int>(slot % a.runs);
  if (row >= a.rows || (a.finished != nullptr && a.finished[row] != 0)) return;
  const T* base = static_cast<const T*>(a.logits) + row * a.row_stride;
  const int step0 = static_cast<int>(static_cast<int64_t>(run) * a.steps / a.runs);
  const int step1 = static_cast<int>(static_cast<int64_t>(run + 1) * a.steps / a.runs);
  auto begin = [&](int step) { return step * kStep<T> + lane * kPer; };            // of the lane's word 0
  float* maxima = a.maxima + static_cast<int64_t>(row) * a.steps;
  float top = -INFINITY, sum = 0.f;
  Held<T> x, next;
  load_step<T, BYTES>(base, begin(step0), a.vocab, next);
  for (int step = step0; step < step1; ++step) {
    x = next;
    // the next step's logits are on their way meanwhile
    if (step + 1 < step1) load_step<T, BYTES>(base, begin(step + 1), a.vocab, next);
    float m = fmaxf(fmaxf(x.top(0), x.top(1)), fmaxf(x.top(2), x.top(3)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) maxima[step] = m;
    if (m > top) {               // the same in all lanes
      float f, none;
      exp_of(Two(top - m, 0.f)).get(&f, &none);
      sum *= f;                  // 0 while the maximum is -infinity
      top = m;
    }
    if (top == -INFINITY) {      // nothing but -infinity, or NaN, which a maximum drops
#pragma unroll
      for (int i = 0; i < kEach<T>; ++i)
        if (const float v = x.at(i); v != v) sum = v;
    } else {
      Two sum0(0.f), sum1(0.f);
      const Two shift(-top);
#pragma unroll
      for (int i = 0; i < kEach<T>; i += 4) {
        sum0 = sum0 + exp_of(Two(x.at(i), x.at(i + 1)) + shift);
        sum1 = sum1 + exp_of(Two(x.at(i + 2), x.at(i + 3)) + shift);
      }
      float s0, s1;
      (sum0 + sum1).get(&s0, &s1);
      sum += s0 + s1;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) a.stats[slot] = make_float2(top, sum);        // a NaN or +infinity leaves a sum that is not finite
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

// A beam of a group: what its keys' values are made of.  kDead: no candidates; kDone: one, the end.
enum BeamState : int { kDead, kDone, kLive };
struct Beam {
  double score, top, log_sum;
  float near;             // score - log_sum in 32 bits
  int state;
};

// A candidate of a group: larger values first, then the lower beam, then the lower token.
struct Candidate {
  unsigned long long value;        // sortable; 0: none
  unsigned long long place;        // beam and token
};
__device__ __forceinline__ bool before(const Candidate& a, const Candidate& b) {
  return a.value > b.value || (a.value == b.value && a.place < b.place);
}

// A CTA a group.  Bound by latency: sums, logarithm, maxima, the border's bits (a barrier each), steps, ranks, each
// waiting for the one before: 9.7 us for 4 beams of 32,000, 12.4 for 64 groups of 8 of 131,072.
template <class T, int BYTES>
__global__ void __launch_bounds__(kThreads) join_kernel(const BeamArgs a) {
  constexpr int kPer = BYTES / sizeof(T);
  __shared__ Beam beam[kMaxOut];
  __shared__ int count, blocks, next;
  __shared__ uint32_t top_key;
  __shared__ int counts[2][32];                  // of the border's bits: from the steps, from the logits
  __shared__ int block[kBlocks];                 // step * beams + beam
  __shared__ Candidate list[kStep<__half> + kMaxOut];
  __shared__ Candidate best[kMaxOut];
  static_assert(kList <= kStep<__half> + kMaxOut, "one list for both paths");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = blockIdx.x, n = a.num_out, row0 = group * a.beams;
  grid_dep_wait();
  grid_dep_launch();
  if (tid == 0) count = blocks = top_key = 0;
  if (tid < 64) counts[tid / 32][tid % 32] = 0;
  for (int b = warp; b < a.beams; b += kWarps) {
    const float score = a.scores[row0 + b];
    Beam m = {score, 0.0, 0.0, score, kDead};
    bool bad = !(fabsf(score) < INFINITY) && score != -INFINITY;
    if (a.finished != nullptr && a.finished[row0 + b] != 0) {
      m.state = kDone;
    } else {
      const float2* stats = a.stats + static_cast<int64_t>(row0 + b) * a.runs;
      // the sums of runs in turn, at the maximum so far
      float top = -INFINITY, sum = 0.f;
      bool odd = false;
      for (int s = lane; s < a.runs; s += 32) {
        const float2 t = stats[s];
        odd |= !(t.y < INFINITY);
        const float most = fmaxf(top, t.x);
        if (t.y > 0.f) {               // most is finite
          float was, is;
          exp_of(Two(top - most, t.x - most)).get(&was, &is);
          sum = fmaf(t.y, is, sum * was);
          top = most;
        }
      }
      float most = top;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      if (sum > 0.f) {
        float w, none;
        exp_of(Two(top - most, 0.f)).get(&w, &none);
        sum *= w;
      }
      top = most;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      bad |= __any_sync(0xffffffffu, odd);
      if (!bad && top > -INFINITY) {
        m.top = top;
        m.log_sum = log_of(sum);
        m.near = static_cast<float>(m.score - m.log_sum);
        m.state = kLive;
      }
    }
    if (bad || score == -INFINITY) m.state = kDead;
    if (bad && lane == 0) report_range(a.status);
    if (lane == 0) beam[b] = m;
  }
  __syncthreads();
  // x - M first: logits of any size keep their differences; the logarithm last: what is equal but for
  // rounding in beams of equal sums stays equal
  auto candidate = [&](float x, int token, int b) {
    const Beam& m = beam[b];
    Candidate c;
    c.value = sortable64((m.score + (static_cast<double>(x == 0.f ? 0.f : x) - m.top)) - m.log_sum);      // -0 is 0
    c.place = static_cast<unsigned long long>(b) << 32 | static_cast<uint32_t>(token);
    return c;
  };
  // In 32 bits the value of logit x is off by less than `off`: *low and the result are below and above it.
  auto nearly = [&](float x, int b, float* low) {
    const float near = beam[b].near, d = x - static_cast<float>(beam[b].top);
    const float v = near + d, off = 0x1p-21f * (fabsf(near) + fabsf(d));
    *low = v - off;
    return v + off;
  };
  // The largest logit of a step of a beam; of a finished one the first step has one candidate, as a logit of 0.
  auto maximum = [&](int step, int b) {
    if (beam[b].state == kLive) return a.maxima[static_cast<int64_t>(row0 + b) * a.steps + step];
    return beam[b].state == kDone && step == 0 ? 0.f : -INFINITY;
  };
  const int all = a.beams * a.steps;
  float mine = -INFINITY;
  for (int i = tid; i < all; i += kThreads) {
    // neighbours are of different beams: a thread's maximum is then seldom that of a beam far behind
    const int b = i % a.beams;
    const float x = maximum(i / a.beams, b);
    float low;
    nearly(x, b, &low);
    if (x > -INFINITY) mine = fmaxf(mine, low);
  }
  const uint32_t key = sortable(mine);
  const uint32_t most = __reduce_max_sync(0xffffffffu, key);
  if (lane == 0) atomicMax(&top_key, most);
  float border = unsortable(border_of(0u, 1u << 31, n, n + n / 2, [&](uint32_t t) { return __syncthreads_count(key >= t); }));
  auto list_steps = [&] {
    for (int i = tid; i < all; i += kThreads) {
      const int b = i % a.beams;
      const float x = maximum(i / a.beams, b);
      float low;
      if (x == -INFINITY || nearly(x, b, &low) < border) continue;
      const int at = atomicAdd(&blocks, 1);
      if (at < kBlocks) block[at] = i;
    }
    __syncthreads();
  };
  list_steps();
  // The bits in which the border and the best key are apart: t0, the ones above, and the first of them.
  auto bits_apart = [&](uint32_t* t0) {
    const uint32_t low = sortable(border), apart = low ^ top_key, bit = apart != 0 ? 1u << (31 - __clz(apart)) : 0u;
    *t0 = bit != 0 ? low & ~(2 * bit - 1) : low;
    return bit;
  };
  if (blocks > kBlocks) {
    // Few threads hold the best (of many beams each thread has one beam's steps, so that the best beams' maxima are
    // few), or fewer than n anything at all: the border from the steps themselves.  64 results of 4 groups of 64 beams
    // far apart, 131,072 bf16 logits: 133 us, and 6,700 step by step; of 64 beams of which one is alive, 2^19 fp32
    // logits: 450 and 6,300.
    uint32_t t0;
    int pass = 0;
    const uint32_t bit = bits_apart(&t0);
    border = unsortable(border_of(t0, bit, n, n + n / 2, [&](uint32_t t) {
      int c = 0;
      for (int i = tid; i < all; i += kThreads) {
        const int b = i % a.beams;
        const float x = maximum(i / a.beams, b);
        float low;
        nearly(x, b, &low);
        c += x > -INFINITY && sortable(low) >= t;
      }
      c = __reduce_add_sync(0xffffffffu, c);
      if (lane == 0 && c > 0) atomicAdd(&counts[0][pass], c);
      __syncthreads();
      return counts[0][pass++];
    }));
    if (bit != 0) {
      __syncthreads();
      if (tid == 0) blocks = 0;
      __syncthreads();
      list_steps();
    }
  }
  // f(beam, held logits, token of the lane's word 0) for the warp's blocks
  auto each_block = [&](auto f) {
    for (int j = warp; j < min(blocks, kBlocks); j += kWarps) {
      const int b = block[j] % a.beams, first = block[j] / a.beams * kStep<T> + lane * kPer;
      Held<T> x;
      if (beam[b].state == kLive)
        load_step<T, BYTES>(static_cast<const T*>(a.logits) + (row0 + b) * a.row_stride, first, a.vocab, x);
      f(b, x, first);
    }
  };
  // Logits of beam b below the result have values below t, whatever was rounded (sign -1); from it on, values from
  // t on (sign 1).
  auto logit_of = [&](float t, int b, float sign) {
    const float near = beam[b].near, top = static_cast<float>(beam[b].top);
    return top + (t - near) + sign * 0x1p-21f * (fabsf(top) + fabsf(t) + fabsf(near));
  };
  auto gather = [&] {
    each_block([&](int b, const Held<T>& x, int first) {
      const float from = logit_of(border, b, -1.f);
      uint32_t which = 0;
      if (beam[b].state == kDone) {
        which = lane == 0 && !(0.f < from);
      } else {
#pragma unroll
        for (int i = 0; i < kEach<T>; ++i) which |= !(x.at(i) < from) && x.at(i) > -INFINITY ? 1u << i : 0u;
      }
      // the logits and their places; made candidates below
      for (; which != 0 && *const_cast<volatile int*>(&count) <= kList; which &= which - 1) {
        const int i = __ffs(which) - 1, token = first + i / kPer * (32 * kPer) + i % kPer, at = atomicAdd(&count, 1);
        if (at >= kList) continue;
        list[at].value = beam[b].state == kDone
                             ? key_of(0.f, a.end_token)
                             : key_of(to_float(static_cast<const T*>(a.logits)[(row0 + b) * a.row_stride + token]), token);
        list[at].place = b;
      }
    });
    __syncthreads();
  };
  gather();
  // Few steps (a small vocabulary), or a beam far ahead that has few: the border from the lanes' shares of them,
  auto again = [&] {
    const bool many = blocks <= kBlocks && count > kList;
    __syncthreads();
    if (many) {                    // the same in all threads
      if (tid == 0) count = 0;
      __syncthreads();             // before anyone counts again, whatever lies between
    }
    return many;
  };
  if (again()) {
    mine = -INFINITY;
    each_block([&](int b, const Held<T>& x, int) {
      float m = 0.f, low;
      if (beam[b].state == kLive) m = fmaxf(fmaxf(x.top(0), x.top(1)), fmaxf(x.top(2), x.top(3)));
      else if (lane != 0) m = -INFINITY;
      nearly(m, b, &low);
      if (m > -INFINITY) mine = fmaxf(mine, low);
    });
    const uint32_t key = sortable(mine);
    border = unsortable(border_of(0u, 1u << 31, n, n + n / 2, [&](uint32_t t) { return __syncthreads_count(key >= t); }));
    gather();
  }
  if (again()) {
    // or from the logits themselves
    int pass = 0;
    uint32_t t0;
    const uint32_t bit = bits_apart(&t0);
    border = unsortable(border_of(t0, bit, n, kList / 2, [&](uint32_t t) {
      const float value = unsortable(t);
      int c = 0;
      each_block([&](int b, const Held<T>& x, int) {
        const float least = logit_of(value, b, 1.f);
        if (beam[b].state == kDone) {
          c += lane == 0 && 0.f >= least;
          return;
        }
#pragma unroll
        for (int i = 0; i < kEach<T>; ++i) c += x.at(i) >= least;
      });
      c = __reduce_add_sync(0xffffffffu, c);
      if (lane == 0 && c > 0) atomicAdd(&counts[1][pass], c);
      __syncthreads();
      return counts[1][pass++];
    }));
    gather();
  }
  auto put = [&](int i, const Candidate& c) {
    const int64_t o = static_cast<int64_t>(group) * n + i;
    const int b = static_cast<int>(c.place >> 32);
    a.parents[o] = c.value == 0 ? -1 : row0 + b;
    a.tokens[o] = c.value == 0 ? -1 : static_cast<int>(static_cast<uint32_t>(c.place));
    const unsigned long long bits = (c.value >> 63) ? c.value & ~(1ull << 63) : ~c.value;
    a.out_scores[o] = c.value == 0 ? -INFINITY : static_cast<float>(__longlong_as_double(static_cast<long long>(bits)));
  };
  const Candidate none = {0, 0};
  // ranks list[0 .. found) and gives f(rank, candidate) the first n
  auto ranked = [&](int found, auto f) {
    for (int i = tid; i < found; i += kThreads) {
      const Candidate c = list[i];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < found; ++j) rank += before(list[j], c);
      if (rank < n) f(rank, c);
    }
  };
  int found = count;
  if (blocks <= kBlocks && found <= kList) {
    static_assert(kList <= kThreads, "a candidate a thread");
    Candidate mine = none;
    if (tid < found)
      mine = candidate(key_value(list[tid].value), key_token(list[tid].value), static_cast<int>(list[tid].place));
    // ranking compares all with all: first drop those whose upper half is not among the n largest
    const uint32_t upper = static_cast<uint32_t>(mine.value >> 32);
    bool in = tid < found;
    if (found > 2 * n) {
      const uint32_t t = border_of(0u, 1u << 31, n, n + n / 2, [&](uint32_t t) { return __syncthreads_count(upper >= t); });
      in = in && upper >= t;
    }
    __syncthreads();
    if (tid == 0) count = 0;
    __syncthreads();
    if (in) list[atomicAdd(&count, 1)] = mine;
    __syncthreads();
    found = count;
    ranked(found, put);
    for (int i = found + tid; i < n; i += kThreads) put(i, none);
    return;
  }
  // Many equal ones: in turn the steps that may have something better than the n best so far, each by what its
  // largest logit would be as its first.
  int kept = 0;
  for (int i = 0; i < all; ++i) {
    if (kept == n) {
      if (tid == 0) next = all;
      __syncthreads();
      for (int j = i + tid; j < all; j += kThreads) {
        const int b = j / a.steps, step = j - b * a.steps;
        const float x = maximum(step, b);
        const int token = beam[b].state == kDone ? a.end_token : step * kStep<T>;
        if (x == -INFINITY || !before(candidate(x, token, b), best[n - 1])) continue;
        atomicMin(&next, j);
        break;
      }
      __syncthreads();
      i = next;
      if (i >= all) break;
    }
    const int b = i / a.steps, step = i % a.steps;
    if (maximum(step, b) == -INFINITY) continue;
    __syncthreads();
    if (tid == 0) count = kept;
    if (tid < kept) list[tid] = best[tid];
    __syncthreads();
    const bool done = beam[b].state == kDone;
    const T* base = static_cast<const T*>(a.logits) + (row0 + b) * a.row_stride;
    for (int v = step * kStep<T> + tid; v < min(a.vocab, (step + 1) * kStep<T>); v += kThreads) {
      const float x = done ? 0.f : to_float(base[v]);
      if (x == -INFINITY || (done && v > 0)) continue;
      const Candidate c = candidate(x, done ? a.end_token : v, b);
      if (kept < n || before(c, best[n - 1])) list[atomicAdd(&count, 1)] = c;
    }
    __syncthreads();
    const int here = count;
    if (here == kept) continue;
    ranked(here, [&](int rank, const Candidate& c) { best[rank] = c; });
    kept = min(here, n);
    __syncthreads();
  }
  for (int i = tid; i < n; i += kThreads) put(i, i < kept ? best[i] : none);
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
int steps_of(const smla_beam_params* p) {
  return (p->vocab - 1) / (p->logits_type == SMLA_FLOAT32 ? kStep<float> : kStep<__half>) + 1;
}

// Runs of a row: the split of least modelled time, in half steps of a warp: its steps and half of one for its start,
// times the waves of warps (32 an SM), half of a run, on average, for the last one to end, and the second launch's
// way through a row's runs, 32 at a time.  512 rows of 128 steps: 35.1, 35.2, 35.7, 37.9 and 36.6 us with 4, 6, 8, 12
// and 16 steps a run.
int runs_of(const smla_beam_params* p) {
  const int steps = steps_of(p), rows = p->groups * p->beams;
  constexpr double kSlots = 152 * 32;
  int best = steps;
  double least = 1e300;
  for (const int each : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64}) {
    const int runs = (steps + each - 1) / each;
    const double waves = static_cast<double>(rows) * runs / kSlots;
    const double cost = (2 * each + 1) * (waves > 1. ? waves : 1.) + each + runs / 24.;
    if (cost < least) {
      least = cost;
      best = runs;
    }
  }
  return best;
}

template <class T, int BYTES>
int launch(const BeamArgs& a, cudaStream_t s) {
  const int64_t warps = static_cast<int64_t>(a.rows) * a.runs;
  const int st = done(launch_programmatic(run_kernel<T, BYTES>, dim3(static_cast<unsigned>((warps - 1) / kRunWarps + 1)),
                                          dim3(kRunWarps * 32), 0, s, a));
  if (st != SMLA_OK) return st;
  return done(launch_programmatic(join_kernel<T, BYTES>, dim3(a.rows / a.beams), dim3(kThreads), 0, s, a));
}
// With the widest load that every row's start allows.
template <class T>
int launch(const BeamArgs& a, cudaStream_t s) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.logits) | static_cast<uintptr_t>(a.row_stride) * sizeof(T);
  if (at % 16 == 0) return launch<T, 16>(a, s);
  if constexpr (sizeof(T) == 2) {
    if (at % 4 != 0) return launch<T, 2>(a, s);
  }
  return launch<T, 4>(a, s);
}

size_t lay_out(const smla_beam_params* p, char* base, BeamArgs* a) {
  const size_t rows = static_cast<size_t>(p->groups) * p->beams;
  a->stats = reinterpret_cast<float2*>(base);
  const size_t at = round256(rows * runs_of(p) * sizeof(float2));
  a->maxima = reinterpret_cast<float*>(base + at);
  return at + round256(rows * steps_of(p) * sizeof(float));
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
                p->groups * p->beams, p->beams, p->vocab, p->num_out, steps_of(p), runs_of(p), p->end_token, nullptr};
  if (workspace_bytes < lay_out(p, static_cast<char*>(workspace), &a)) return SMLA_ERR_WORKSPACE_TOO_SMALL;
  st = ready(&a.status);
  if (st != SMLA_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (p->logits_type == SMLA_FLOAT32) return launch<float>(a, s);
  return p->logits_type == SMLA_BFLOAT16 ? launch<__nv_bfloat16>(a, s) : launch<__half>(a, s);
}

}  // extern "C"
