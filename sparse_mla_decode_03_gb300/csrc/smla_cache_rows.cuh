// Where a new token of the paged cache lands and how its row is written, by one warp a token:
// shared by the append with and without the rotation, and by the call that reads rows back.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/smla.h"
#include "smla_internal.h"
#include "smla_ptx.cuh"

namespace smla {

__device__ __forceinline__ void report(int* status, int code) { atomicCAS(status, 0, code); }

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

// Sequence and position of token t.  b = -1 outside every sequence; a position may be negative.
struct Place {
  int b;
  int64_t pos;
};
__device__ __forceinline__ Place place_of(const AppendArgs& a, int t) {
  Place p = {sequence_of(a.cu_q, a.B, t), 0};
  if (p.b >= 0) p.pos = static_cast<int64_t>(__ldg(a.kv_lens + p.b)) - (__ldg(a.cu_q + p.b + 1) - t);
  return p;
}

// The row of a place, or null (reported) if it has none; null too outside every sequence.
__device__ __forceinline__ uint8_t* row_at(const AppendArgs& a, const Place& p) {
  if (p.b < 0) return nullptr;
  if (p.pos >= 0) {   // below 2^31: kv_lens is an int32
    const uint32_t at = static_cast<uint32_t>(p.pos), page = at / static_cast<uint32_t>(a.page_size);
    if (page < static_cast<uint32_t>(a.max_pages)) {
      const int phys = __ldg(a.table + static_cast<int64_t>(p.b) * a.max_pages + page);
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

// Largest magnitude of a lane's 16 columns as bf16 bits, two columns at a time (magnitudes compare
// as integers).
__device__ __forceinline__ uint32_t top_of(const uint32_t (&w)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_u16x2(m, w[i] & 0x7fff7fffu);
  return max(m >> 16, m & 0xffffu);
}

// One token of a warp.  Lane l < 28 holds nope columns 16 l .. 16 l + 15 (four lanes a scale
// group), lanes 28..31 the rope.  The row is put together in shared memory (stage: 73 words)
// and leaves in consecutive words.
__device__ __forceinline__ void write_row(const AppendArgs& a, uint8_t* dst, const uint4& u0, const uint4& u1,
                                          uint2* stage) {
  const int lane = threadIdx.x & 31;
  uint32_t w[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
  uint32_t top = top_of(w);
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

// Four words of 8 columns' e2m1 nibbles: column 2 p of a word in nibble p, column 2 p + 1 in nibble
// p + 4, so that one shift of a word brings a pair of neighbours to the two halves of a bf16 pair.
__device__ __forceinline__ uint32_t pack_e2m1(const uint32_t* w, float inv) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16) * inv;
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u) * inv;
  }
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %3, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %7, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %4, %2;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %6;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// The same for a row of 4-bit values (two lanes a scale group of 32 columns).  stage: 23 16-byte words.
__device__ __forceinline__ void write_row4(const AppendArgs& a, uint8_t* dst, const uint4& u0, const uint4& u1,
                                           uint4* stage) {
  const int lane = threadIdx.x & 31;
  uint32_t w[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
  uint32_t top = top_of(w);
  const uint32_t other = __shfl_xor_sync(0xffffffffu, top, 1);
  top = max(top, other);
  const bool bad = top >= 0x7f80u;       // infinity or NaN: there is no such nibble, the scale says it
  // 6 = 1.5 * 2^2, so the least e with top <= 6 * 2^e follows from top's exponent and whether its
  // mantissa exceeds 1.5: exact, no logarithm.
  int byte = static_cast<int>(top >> 7) - 2 + ((top & 0x7fu) > 0x40u ? 1 : 0);
  byte = top == 0 ? 127 : max(byte, 1);                  // 253 at most
  // from 1.75 * 2^127 on (halfway from 3 to 4 in the scale 2^126) the stored value is 2^128
  if (lane < 28 && top >= 0x7f60u) report(a.status, SMLA_ERR_RANGE);
  const float inv = bad ? 0.f : __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);
  uint8_t* bytes = reinterpret_cast<uint8_t*>(stage);
  if (lane < 28) {
    if (bad) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 0;
    }
    reinterpret_cast<uint2*>(stage)[lane] = make_uint2(pack_e2m1(w, inv), pack_e2m1(w + 4, inv));
    if ((lane & 1) == 0) bytes[kRow4Scales + lane / 2] = static_cast<uint8_t>(bad ? 255 : byte);
  } else {
    uint4* d = stage + kRow4Rope / 16 + 2 * (lane - 28);
    d[0] = u0;
    d[1] = u1;
    if (lane == 28) *reinterpret_cast<uint16_t*>(bytes + kRow4Rope - 2) = 0;     // the padding
  }
  __syncwarp();
  if (lane < kRow4Bytes / 16) reinterpret_cast<uint4*>(dst)[lane] = stage[lane];
  __syncwarp();
}

// ---------------------------------------------------------------------------
// Reading rows
// ---------------------------------------------------------------------------
__device__ __forceinline__ float ue8m0_value(uint32_t e) {
  return __uint_as_float(e == 0u ? 0x00400000u : (e == 255u ? 0x7fffffffu : (e << 23)));
}

// 16 columns of nope (lanes 0..27: 16 l ..) or rope (lanes 28..31) of a row as eight bf16 pairs.  Its loads
// and the arithmetic are apart, so that a caller has several rows on their way.
struct RowLane {
  uint2 v[4];
  uint32_t scale;
};
template <bool ROW4>
__device__ __forceinline__ void load_row(const uint8_t* src, RowLane& d) {
  const int lane = threadIdx.x & 31;
  d.v[0] = d.v[1] = d.v[2] = d.v[3] = make_uint2(0u, 0u);
  d.scale = 127;
  if (src == nullptr) return;
  if (lane >= 28) {
    const uint2* w = reinterpret_cast<const uint2*>(src + (ROW4 ? kRow4Rope : 456) + 32 * (lane - 28));
#pragma unroll
    for (int k = 0; k < 4; ++k) d.v[k] = __ldg(w + k);
  } else if (ROW4) {
    d.v[0] = __ldg(reinterpret_cast<const uint2*>(src) + lane);
    d.scale = __ldg(src + kRow4Scales + lane / 2);
  } else {
    d.v[0] = __ldg(reinterpret_cast<const uint2*>(src) + 2 * lane);
    d.v[1] = __ldg(reinterpret_cast<const uint2*>(src) + 2 * lane + 1);
    d.scale = __ldg(src + kNope + lane / 4);
  }
}
// e4m3 (by way of f16, exact) or e2m1 times a power of two.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t two, float scale) {
  uint32_t h2;
  const uint16_t in = static_cast<uint16_t>(two);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(in));
  float lo, hi;
  asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;}" : "=f"(lo), "=f"(hi) : "r"(h2));
  return pack_bf16(lo * scale, hi * scale);
}
// Nibble n of w, its exponent and mantissa in a float's lowest exponent bits: its value times 2^-126,
// subnormals included, so two exact products put both powers right.
__device__ __forceinline__ float e2m1_value(uint32_t w, int n, float scale) {
  const uint32_t c = w >> (4 * n);
  return __uint_as_float((c & 8u) << 28 | (c & 7u) << 22) * 0x1p126f * scale;
}
template <bool ROW4>
__device__ __forceinline__ void row_values(const RowLane& d, uint32_t (&o)[8]) {
  const int lane = threadIdx.x & 31;
  if (lane >= 28) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      o[2 * k] = d.v[k].x;
      o[2 * k + 1] = d.v[k].y;
    }
    return;
  }
  const float f = ue8m0_value(d.scale);
  if (ROW4) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t w = k < 4 ? d.v[0].x : d.v[0].y;
      o[k] = pack_bf16(e2m1_value(w, k & 3, f), e2m1_value(w, (k & 3) + 4, f));
    }
  } else {
    const uint32_t w[4] = {d.v[0].x, d.v[0].y, d.v[1].x, d.v[1].y};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      o[2 * k] = e4m3_pair(w[k] & 0xffffu, f);
      o[2 * k + 1] = e4m3_pair(w[k] >> 16, f);
    }
  }
}

}  // namespace smla
