// Attention of a chunk of new tokens over the paged cache (smla_chunk_attention).
// Declared and documented in include/smla.h.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/smla.h"
#include "smla_internal.h"
#include "smla_ptx.cuh"

namespace smla {
namespace {

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
};

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  uint32_t h2;
  const uint16_t in = static_cast<uint16_t>(byte);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(in));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h2 & 0xffffu)));
}
__device__ __forceinline__ float ue8m0_value(uint32_t e) {
  return __uint_as_float(e == 0u ? 0x00400000u : (e == 255u ? 0x7fffffffu : (e << 23)));
}

// One CTA per (token, head), element-wise fp32: four warps take the visible positions in
// turn, each with its own online softmax, merged at the end.
__global__ void __launch_bounds__(128) chunk_plain_kernel(const ChunkArgs a) {
  __shared__ float qs[kQkDim];
  __shared__ float wm[4], wl[4];
  __shared__ float wacc[4][kNope];
  grid_dep_wait();
  grid_dep_launch();
  const int h = blockIdx.y, t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (t < a.cu_q[0] || t >= a.cu_q[a.B]) return;
  int b = 0;
  for (int hi = a.B; hi - b > 1;) {
    const int mid = (b + hi) / 2;
    if (a.cu_q[mid] <= t) b = mid;
    else hi = mid;
  }
  const int len = a.kv_lens[b];
  const int pos = len - (a.cu_q[b + 1] - t);
  const int lo = a.vis_begin ? max(0, a.vis_begin[t]) : 0;
  const int hi = a.vis_end ? min(len, a.vis_end[t]) : pos + 1;
  const uint16_t* qrow = a.q + (static_cast<int64_t>(t) * a.H + h) * kQkDim;
  for (int c = threadIdx.x; c < kQkDim; c += blockDim.x)
    qs[c] = __uint_as_float(static_cast<uint32_t>(qrow[c]) << 16);
  __syncthreads();
  float m = -INFINITY, l = 0.f;
  float acc[16];
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  for (int s = lo + warp; s < hi; s += 4) {
    const int page = s / a.page_size;
    if (page >= a.max_pages) {
      if (lane == 0) atomicCAS(a.status, 0, SMLA_ERR_INDEX_RANGE);
      continue;
    }
    const int phys = a.table[static_cast<int64_t>(b) * a.max_pages + page];
    if (phys < 0) continue;
    const int64_t r = static_cast<int64_t>(phys) * a.page_size + s % a.page_size;
    if (r >= a.num_rows) {
      if (lane == 0) atomicCAS(a.status, 0, SMLA_ERR_INDEX_RANGE);
      continue;
    }
    const uint8_t* row = a.pool + r * a.stride;
    float v[16];
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int w = lane + 32 * j;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * j + e] = 0.f;
      if (w < kNope / 4) {
        const uint32_t word = __ldg(reinterpret_cast<const uint32_t*>(row) + w);
        const float sc = ue8m0_value(__ldg(row + kNope + (4 * w) / 64));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[4 * j + e] = e4m3_value((word >> (8 * e)) & 0xffu) * sc;
          dot = fmaf(qs[4 * w + e], v[4 * j + e], dot);
        }
      }
    }
    const uint32_t rw = __ldg(reinterpret_cast<const uint32_t*>(row + 456) + lane);
    dot = fmaf(qs[kNope + 2 * lane], __uint_as_float(rw << 16), dot);
    dot = fmaf(qs[kNope + 2 * lane + 1], __uint_as_float(rw & 0xffff0000u), dot);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    float x = dot * a.scale;
    if (a.cap > 0.f) x = a.cap * tanhf(x / a.cap);
    if (a.slopes) x -= a.slopes[h] * fabsf(static_cast<float>(pos - s));
    const float m_new = fmaxf(m, x);
    const float f = expf(m - m_new), p = expf(x - m_new);
    l = l * f + p;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = acc[i] * f + p * v[i];
    m = m_new;
  }
  if (lane == 0) {
    wm[warp] = m;
    wl[warp] = l;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int w = lane + 32 * j;
    if (w < kNope / 4) {
#pragma unroll
      for (int e = 0; e < 4; ++e) wacc[warp][4 * w + e] = acc[4 * j + e];
    }
  }
  __syncthreads();
  const float M = fmaxf(fmaxf(wm[0], wm[1]), fmaxf(wm[2], wm[3]));
  float L = 0.f, fw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    fw[i] = wm[i] == -INFINITY ? 0.f : expf(wm[i] - M);
    L += wl[i] * fw[i];
  }
  const float inv = L > 0.f ? 1.f / L : 0.f;
  __nv_bfloat16* orow = a.out + (static_cast<int64_t>(t) * a.H + h) * kNope;
  for (int c = threadIdx.x; c < kNope; c += blockDim.x)
    orow[c] = __float2bfloat16_rn((wacc[0][c] * fw[0] + wacc[1][c] * fw[1] + wacc[2][c] * fw[2] +
                                   wacc[3][c] * fw[3]) * inv);
  if (threadIdx.x == 0) a.lse[static_cast<int64_t>(t) * a.H + h] = L > 0.f ? M + logf(L) : -INFINITY;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_chunk(const smla_chunk_params* p) {
  if (p == nullptr || p->reserved != 0) return SMLA_ERR_INVALID_ARG;
  if (p->batch < 1 || p->total_q < 1 || p->page_size < 1 || p->max_pages < 1 || p->num_rows < 1 ||
      p->max_kv_tokens < 1)
    return SMLA_ERR_INVALID_ARG;
  if (p->kv_row_stride < kRowBytes || p->kv_row_stride % 8 != 0) return SMLA_ERR_INVALID_ARG;
  if (!(std::isfinite(p->softmax_scale) && p->softmax_scale > 0.f)) return SMLA_ERR_INVALID_ARG;
  if (!(std::isfinite(p->logit_cap) && p->logit_cap >= 0.f)) return SMLA_ERR_INVALID_ARG;
  if (p->num_heads != 16 && p->num_heads != 32 && p->num_heads != 64 && p->num_heads != 128)
    return SMLA_ERR_UNSUPPORTED_SHAPE;
  if (p->batch > 65535 || static_cast<int64_t>(p->total_q) * p->num_heads >= (int64_t{1} << 30))
    return SMLA_ERR_UNSUPPORTED_SHAPE;
  return SMLA_OK;
}

}  // namespace
}  // namespace smla

using namespace smla;   // NOLINT: the entry points below are this file's own

extern "C" {

int smla_chunk_workspace_size(const smla_chunk_params* p, size_t* bytes) {
  const int st = check_chunk(p);
  if (st != SMLA_OK) return st;
  if (bytes == nullptr) return SMLA_ERR_INVALID_ARG;
  *bytes = 256;
  return SMLA_OK;
}

int smla_chunk_attention(const void* q, const void* kv_pages, const int32_t* block_table,
                         const int32_t* cu_q, const int32_t* kv_lens, const int32_t* vis_begin,
                         const int32_t* vis_end, const float* slopes, void* out, float* lse,
                         const smla_chunk_params* p, void* workspace, size_t workspace_bytes,
                         smla_stream_t stream) {
  int st = check_chunk(p);
  if (st != SMLA_OK) return st;
  if (q == nullptr || kv_pages == nullptr || block_table == nullptr || cu_q == nullptr ||
      kv_lens == nullptr || out == nullptr || lse == nullptr || workspace == nullptr)
    return SMLA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv_pages, 16) || !aligned(out, 16) || !aligned(workspace, 256) ||
      !aligned(block_table, 4) || !aligned(cu_q, 4) || !aligned(kv_lens, 4) || !aligned(vis_begin, 4) ||
      !aligned(vis_end, 4) || !aligned(slopes, 4) || !aligned(lse, 4))
    return SMLA_ERR_INVALID_ARG;
  size_t need = 0;
  st = smla_chunk_workspace_size(p, &need);
  if (st != SMLA_OK) return st;
  if (workspace_bytes < need) return SMLA_ERR_WORKSPACE_TOO_SMALL;
  st = check_device();
  if (st != SMLA_OK) return st;
  int* status = nullptr;
  if (status_word_address(&status) != cudaSuccess) return SMLA_ERR_CUDA;
  const ChunkArgs a = {static_cast<const uint16_t*>(q), static_cast<const uint8_t*>(kv_pages),
                       block_table, cu_q, kv_lens, vis_begin, vis_end, slopes,
                       static_cast<__nv_bfloat16*>(out), lse, p->batch, p->num_heads, p->total_q,
                       p->page_size, p->max_pages, p->num_rows, p->kv_row_stride, p->softmax_scale,
                       p->logit_cap, status};
  const cudaError_t e = launch_programmatic(chunk_plain_kernel, dim3(p->total_q, p->num_heads), dim3(128), 0,
                                            reinterpret_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

}  // extern "C"
