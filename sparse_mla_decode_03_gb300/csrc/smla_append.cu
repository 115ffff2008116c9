// Writing new tokens into the paged cache, with or without the position rotation on the way
// (smla_cache_append, smla_cache_append_rotary), and reading them back (smla_cache_read).
// Declared and documented in include/smla.h.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/smla.h"
#include "smla_cache_host.h"
#include "smla_cache_rows.cuh"
#include "smla_internal.h"
#include "smla_ptx.cuh"

namespace smla {
namespace {

template <bool ROW4>
__device__ __forceinline__ void write_any(const AppendArgs& a, uint8_t* dst, const uint4& u0, const uint4& u1,
                                          uint4* stage) {
  if (ROW4) write_row4(a, dst, u0, u1, stage);
  else write_row(a, dst, u0, u1, reinterpret_cast<uint2*>(stage));
}

// Bound by memory: 1,024 bytes in and 584 out a token.  One token a warp: 38 us for 131,072 tokens
// (5.55 TB/s, 82 % of the measured copy rate; issue 73 %, integer pipe 59 % busy); two or four
// tokens' loads at once measured 41.0 and 44.1 us.  A decode step's call (96 tokens) is a launch
// and two trips to memory, 5 us.
template <bool ROW4>
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs a) {
  __shared__ uint4 stage[8][38];
  grid_dep_wait();
  grid_dep_launch();
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= a.total) return;
  const uint4* src = a.kv + t * a.token_units + 2 * (threadIdx.x & 31);
  const uint4 u0 = __ldcs(src), u1 = __ldcs(src + 1);
  uint8_t* dst = row_at(a, place_of(a, t));
  if (dst != nullptr) write_any<ROW4>(a, dst, u0, u1, stage[threadIdx.x >> 5]);
}

// ---------------------------------------------------------------------------
// Rotation
// ---------------------------------------------------------------------------
struct RotaryArgs {
  const float* turn;            // [rows][64]: cosines of the 32 pairs, sines
  int64_t rows;
  const uint4* q_rope;          // null: no queries
  uint4* q;                     // its column 448
  int64_t qr_token, qr_head, q_token, q_head;     // 16-byte units
  int H, chunks;                // chunks: of kHeads heads
};
constexpr int kHeads = 16;      // of a token's queries that a warp rotates

__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Cosines and sines of the pairs in 8 columns from 8 * unit on: pairs of neighbours (4 of them) or
// of columns i and i + 32 (8).
template <bool NEIGHBOURS>
struct Turn {
  static constexpr int kPairs = NEIGHBOURS ? 4 : 8;
  float c[kPairs], s[kPairs];
  __device__ __forceinline__ Turn(const float* turn, int unit) {
    const float4* from = reinterpret_cast<const float4*>(turn) + (NEIGHBOURS ? unit : 2 * (unit & 3));
#pragma unroll
    for (int k = 0; k < kPairs / 4; ++k) {
      const float4 x = __ldg(from + k), y = __ldg(from + 8 + k);
      c[4 * k] = x.x, c[4 * k + 1] = x.y, c[4 * k + 2] = x.z, c[4 * k + 3] = x.w;
      s[4 * k] = y.x, s[4 * k + 1] = y.y, s[4 * k + 2] = y.z, s[4 * k + 3] = y.w;
    }
  }
  // (a, b) -> (a c - b s, a s + b c), in 32 bits, rounded to bf16 once.  For pairs 32 apart `other` are
  // the partner's columns and upper tells which of the two this is.
  __device__ __forceinline__ uint4 operator()(const uint4& x, const uint4& other, bool upper) const {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w}, v[4] = {other.x, other.y, other.z, other.w};
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (NEIGHBOURS) {
        const float a = low(w[k]), b = high(w[k]);
        o[k] = pack_bf16(fmaf(a, c[k], -(b * s[k])), fmaf(a, s[k], b * c[k]));
      } else {
        const float s0 = upper ? s[2 * k] : -s[2 * k], s1 = upper ? s[2 * k + 1] : -s[2 * k + 1];
        o[k] = pack_bf16(fmaf(low(w[k]), c[2 * k], low(v[k]) * s0), fmaf(high(w[k]), c[2 * k + 1], high(v[k]) * s1));
      }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
};

__device__ __forceinline__ uint4 shfl_xor(const uint4& x, int mask) {
  return make_uint4(__shfl_xor_sync(0xffffffffu, x.x, mask), __shfl_xor_sync(0xffffffffu, x.y, mask),
                    __shfl_xor_sync(0xffffffffu, x.z, mask), __shfl_xor_sync(0xffffffffu, x.w, mask));
}

// A warp takes a token's row, or the rope columns of kHeads of its queries (8 lanes a head, 16 bytes a lane,
// each of which a lane reads before it writes there, and no other lane: q_rope may be q's own columns).  Bound by
// memory: 16 heads a token are 2,048 bytes in and out beside the row's 1,608; 65,536 tokens take 62 us (374 MB, 6.0
// TB/s, 89 % of the measured copy rate).  Products and sums in 32 bits, one rounding to bf16, so that a rotation by
// nothing changes no finite value but a zero's sign (beside a partner below 0).  A step's call (96 tokens of 64 heads) is a launch and three trips to memory (offsets,
// lengths, then the table's row), 5 us.
template <bool ROW4, bool NEIGHBOURS>
__global__ void __launch_bounds__(256) append_rotary_kernel(const AppendArgs a, const RotaryArgs r) {
  __shared__ uint4 stage[8][38];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t item = blockIdx.x * 8u + warp, per = 1u + r.chunks, tok = item / per, chunk = item - tok * per;
  if (tok >= static_cast<uint32_t>(a.total)) return;
  const int t = static_cast<int>(tok);
  if (chunk == 0) {
    const uint4* src = a.kv + t * a.token_units + 2 * lane;
    uint4 u0 = __ldcs(src), u1 = __ldcs(src + 1);
    const Place p = place_of(a, t);
    if (p.b < 0) return;
    if (p.pos < 0 || p.pos >= r.rows) {
      if (lane == 0) report(a.status, SMLA_ERR_INDEX_RANGE);
      return;
    }
    uint8_t* dst = row_at(a, p);
    if (dst == nullptr) return;
    // lanes 28..31 hold the rope, 16 columns each
    const int unit = 2 * (lane & 3);
    const float* turn = r.turn + p.pos * 64;
    const Turn<NEIGHBOURS> t0(turn, unit), t1(turn, unit + 1);
    const uint4 v0 = NEIGHBOURS ? u0 : shfl_xor(u0, 2), v1 = NEIGHBOURS ? u1 : shfl_xor(u1, 2);
    if (lane >= 28) {
      u0 = t0(u0, v0, unit >= 4);
      u1 = t1(u1, v1, unit >= 4);
    }
    write_any<ROW4>(a, dst, u0, u1, stage[warp]);
    return;
  }
  const int unit = lane & 7, h0 = static_cast<int>(chunk - 1) * kHeads + lane / 8;
  const uint4* src = r.q_rope + t * r.qr_token + unit;
  uint4 x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    x[k] = h0 + 4 * k < r.H ? __ldcs(src + (h0 + 4 * k) * r.qr_head) : make_uint4(0u, 0u, 0u, 0u);
  const Place p = place_of(a, t);
  if (p.b < 0 || p.pos < 0 || p.pos >= r.rows) return;      // reported with the token's row
  const Turn<NEIGHBOURS> turn(r.turn + p.pos * 64, unit);
  uint4* dst = r.q + t * r.q_token + unit;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint4 y = turn(x[k], NEIGHBOURS ? x[k] : shfl_xor(x[k], 4), unit >= 4);
    if (h0 + 4 * k < r.H) dst[(h0 + 4 * k) * r.q_head] = y;
  }
}

// ---------------------------------------------------------------------------
// Reading back
// ---------------------------------------------------------------------------
// A token a warp, 368 or 584 bytes in and 1,024 out; the products are exact, but at the ends of bf16's
// range.  10,005 tokens of 4-bit rows: 7.5 us (14 MB), a launch and three trips to memory.
template <bool ROW4>
__global__ void __launch_bounds__(256) read_kernel(const AppendArgs a, uint4* out, int64_t out_units) {
  grid_dep_wait();
  grid_dep_launch();
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (t >= a.total) return;
  const uint8_t* src = row_at(a, place_of(a, t));
  if (src == nullptr) return;
  RowLane d;
  load_row<ROW4>(src, d);
  uint32_t o[8];
  row_values<ROW4>(d, o);
  uint4* dst = out + t * out_units + 2 * lane;
  dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
  dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

int check_tokens(const void* kv, int64_t kv_token_stride, int32_t total_tokens, const void* kv_pages,
                 const int32_t* block_table, const int32_t* cu_q, const int32_t* kv_lens,
                 const smla_cache_params* c) {
  const int st = check_cache(c);
  if (st != SMLA_OK) return st;
  if (total_tokens < 0 || kv_token_stride < kQkDim || kv_token_stride % 8 != 0)
    return SMLA_ERR_INVALID_ARG;
  if (!pool_ok(kv_pages, c) || !ints_ok(block_table) || !ints_ok(cu_q) || !ints_ok(kv_lens))
    return SMLA_ERR_INVALID_ARG;
  return total_tokens > 0 && (kv == nullptr || !aligned(kv, 16)) ? SMLA_ERR_INVALID_ARG : SMLA_OK;
}
AppendArgs append_args(const void* kv, int64_t kv_token_stride, int32_t total_tokens, const void* kv_pages,
                       const int32_t* block_table, const int32_t* cu_q, const int32_t* kv_lens,
                       const smla_cache_params* c, int* status) {
  return {static_cast<const uint4*>(kv), kv_token_stride / 8, total_tokens,
          static_cast<uint8_t*>(const_cast<void*>(kv_pages)), block_table, cu_q, kv_lens, c->num_seqs,
          c->max_pages, c->page_size, c->num_pages, c->kv_row_stride, status};
}
dim3 warps(int64_t items) { return dim3(static_cast<unsigned>((items - 1) / 8 + 1)); }

}  // namespace
}  // namespace smla

using namespace smla;   // NOLINT: the entry points below are this file's own

extern "C" {

int smla_cache_append(const void* kv, int64_t kv_token_stride, int32_t total_tokens, void* kv_pages,
                      const int32_t* block_table, const int32_t* cu_q, const int32_t* kv_lens,
                      const smla_cache_params* c, smla_stream_t stream) {
  int st = check_tokens(kv, kv_token_stride, total_tokens, kv_pages, block_table, cu_q, kv_lens, c);
  if (st != SMLA_OK || total_tokens == 0) return st;
  int* status = nullptr;
  st = ready(&status);
  if (st != SMLA_OK) return st;
  const AppendArgs a = append_args(kv, kv_token_stride, total_tokens, kv_pages, block_table, cu_q, kv_lens, c, status);
  return done(launch_programmatic(is_row4(c->kv_row_stride) ? append_kernel<true> : append_kernel<false>,
                                  warps(total_tokens), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), a));
}

int smla_cache_append_rotary(const void* kv, int64_t kv_token_stride, int32_t total_tokens, void* kv_pages,
                             const int32_t* block_table, const int32_t* cu_q, const int32_t* kv_lens,
                             const smla_cache_params* c, const smla_rotary_params* r, smla_stream_t stream) {
  int st = check_tokens(kv, kv_token_stride, total_tokens, kv_pages, block_table, cu_q, kv_lens, c);
  if (st != SMLA_OK) return st;
  if (r == nullptr || r->table == nullptr || !aligned(r->table, 16) || r->table_rows < 1 || r->reserved != 0 ||
      (r->pairing != SMLA_ROTARY_NEIGHBOURS && r->pairing != SMLA_ROTARY_HALVES) || r->num_heads < 0)
    return SMLA_ERR_INVALID_ARG;
  if (r->num_heads > 0) {
    if (r->q_rope_token_stride % 8 != 0 || r->q_rope_head_stride % 8 != 0 || r->q_token_stride % 8 != 0 ||
        r->q_head_stride % 8 != 0 || r->q_rope_token_stride < 0 || r->q_rope_head_stride < 0 ||
        r->q_token_stride < 0 || r->q_head_stride < 0)
      return SMLA_ERR_INVALID_ARG;
    if (total_tokens > 0 && (r->q_rope == nullptr || r->q == nullptr || !aligned(r->q_rope, 16) || !aligned(r->q, 16)))
      return SMLA_ERR_INVALID_ARG;
  }
  const int64_t chunks = (static_cast<int64_t>(r->num_heads) + kHeads - 1) / kHeads;
  if (total_tokens * (1 + chunks) >= (int64_t{1} << 31)) return SMLA_ERR_UNSUPPORTED_SHAPE;
  if (total_tokens == 0) return SMLA_OK;
  int* status = nullptr;
  st = ready(&status);
  if (st != SMLA_OK) return st;
  const AppendArgs a = append_args(kv, kv_token_stride, total_tokens, kv_pages, block_table, cu_q, kv_lens, c, status);
  const RotaryArgs ra = {r->table, r->table_rows, static_cast<const uint4*>(r->q_rope),
                         static_cast<uint4*>(r->q) + kNope / 8, r->q_rope_token_stride / 8,
                         r->q_rope_head_stride / 8, r->q_token_stride / 8, r->q_head_stride / 8, r->num_heads,
                         static_cast<int>(chunks)};
  const bool four = is_row4(c->kv_row_stride), next = r->pairing == SMLA_ROTARY_NEIGHBOURS;
  return done(launch_programmatic(four ? (next ? append_rotary_kernel<true, true> : append_rotary_kernel<true, false>)
                                       : (next ? append_rotary_kernel<false, true> : append_rotary_kernel<false, false>),
                                  warps(total_tokens * (1 + chunks)), dim3(256), 0,
                                  reinterpret_cast<cudaStream_t>(stream), a, ra));
}

int smla_cache_read(const void* kv_pages, const int32_t* block_table, const int32_t* cu_q, const int32_t* kv_lens,
                    void* out, int64_t out_token_stride, int32_t total_tokens, const smla_cache_params* c,
                    smla_stream_t stream) {
  int st = check_tokens(out, out_token_stride, total_tokens, kv_pages, block_table, cu_q, kv_lens, c);
  if (st != SMLA_OK || total_tokens == 0) return st;
  int* status = nullptr;
  st = ready(&status);
  if (st != SMLA_OK) return st;
  const AppendArgs a = append_args(nullptr, kQkDim, total_tokens, kv_pages, block_table, cu_q, kv_lens, c, status);
  return done(launch_programmatic(is_row4(c->kv_row_stride) ? read_kernel<true> : read_kernel<false>,
                                  warps(total_tokens), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), a,
                                  static_cast<uint4*>(out), out_token_stride / 8));
}

}  // extern "C"
