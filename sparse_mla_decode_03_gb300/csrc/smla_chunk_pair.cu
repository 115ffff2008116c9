// Chunk attention on pairs of SMs: the kernel for many query rows.
//
// The (token, head) rows of a sequence are cut into tiles of 256; all heads share K and V
// (k = the 512-wide row, v = its first 448 columns), so a tile is a plain matrix problem:
// S = Q K^T (256 x 64 x 512 a block of 64 positions), O += P V (256 x 448 x 64).
//
// What bounds it.  The tensor core needs 1,920 cycles a block (4,096 multiply-adds a
// cycle and SM), and shared memory feeds it 128 bytes a cycle: with one SM on 128 rows,
// Q alone (128 KB a block) would take as long as its product, and the same block of K and
// V would be read by every SM.  A pair (tcgen05 cta_group::2) works on 256 rows: each SM
// keeps half of the rows (Q, S, P, O) and brings half of the other operand, 32 of the 64
// positions for K and half of the columns for V.  That is 80 KB of Q and K for 1,024
// cycles of the first product (1,280 cycles of shared memory) and 60 KB of P and V for 896
// of the second: together about 2,400 cycles a block with the incoming copies.
// Tensor memory is full: O takes 448 columns, S the other 64.  So there is one S; the
// softmax takes it into registers at once and P goes through shared memory, which
// lets the scores of block i + 1 run while the softmax of block i does.
//
// K and V are read from an expanded copy (bf16 rows, the e4m3 values times their
// powers of two: exact), which a kernel before this one writes once a call: 1.6 KB moved a
// position, against 960 multiply-adds for each of its query rows.
//
// Measured: 1,024 tokens of 128 heads behind 15,360 positions in 2.22 ms with plan, expansion
// and merge, 1.80 PFLOP/s (93 % of the measured matrix rate); 512 tokens of 64 heads in 8,192
// positions 278 of 310 us, tensor pipe 78 % busy, the tensor core's shared-memory reads 69 %.
// The issuing warp walks its schedule as one and elects a lane for the products alone: issued
// by a branch of one lane they took 87 cycles each, against 45 to 64.
//
// Warps of a CTA: 0..3 softmax and results (a thread a row), 4 tensor copies (one lane), 5
// in the leading CTA issues the products.  Every wait is bounded.
#include <cstring>
#include <mutex>

#include "smla_chunk.h"
#include "smla_chunk_rows.cuh"
#include "smla_ptx.cuh"

namespace smla {
namespace {

constexpr int kThreads = 192;
constexpr int kStages = 5;
constexpr int kStage = 16384;      // K: 32 positions x 256 columns; V: 64 positions x 128 columns
constexpr int kQBytes = 128 * 1024;
constexpr int kRingOff = kQBytes;
constexpr int kPOff = kRingOff + kStages * kStage;
constexpr int kBarOff = kPOff + 128 * 128;
constexpr int kSmem = kBarOff + 512 + 1024;
constexpr uint32_t kColS = 448;
// FULL: a stage's copies have landed in both CTAs (the leader's counts); EMPTY: the
// products that read a stage are done; QFULL / QEMPTY: the same of Q; SFULL: the scores
// of a block are in tensor memory; SEMPTY: both CTAs' softmax have taken them (leader);
// PFULL: both have written P (leader); PV: the value product of a block is done; OEMPTY:
// both have taken O (leader).
enum Bar : int { FULL = 0, EMPTY = FULL + kStages, QFULL = EMPTY + kStages, QEMPTY, SFULL, SEMPTY, PFULL, PV, OEMPTY, kBars };

struct Maps {
  CUtensorMap q, k, v;
};

template <bool MODS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    pair_kernel(const ChunkArgs a, const ChunkPlan plan, const __grid_constant__ Maps maps) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int worker = blockIdx.x >> 1;
  auto bar = [&](int i) { return sbase + kBarOff + 8u * static_cast<uint32_t>(i); };
  volatile uint32_t* taddr = reinterpret_cast<volatile uint32_t*>(smem + kBarOff + 8 * kBars);
  volatile int* stop = reinterpret_cast<volatile int*>(smem + kBarOff + 8 * kBars + 8);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBars; ++i)
      mbar_init(bar(i), i == SEMPTY || i == PFULL || i == OEMPTY ? 8 : 1);
    *stop = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc_pair(sbase + kBarOff + 8 * kBars, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive_wait();
  tc_fence_after();
  const uint32_t tmem = *taddr;
  grid_dep_wait();
  grid_dep_launch();

  const int t_first = plan.start[worker], x0 = plan.begin[worker], x1 = plan.begin[worker + 1];

  if (warp == 4) {
    // ---------------- tensor copies ----------------
    if (lane == 0) {
      uint32_t n = 0;            // stages filled
      uint32_t nq = 0;
      bool ok = true;
      const uint32_t full0 = dsmem_addr(bar(FULL), 0), qfull = dsmem_addr(bar(QFULL), 0);
      auto stage = [&](uint32_t* dst) {       // the next free stage
        const uint32_t s = n % kStages, use = n / kStages;
        if (use > 0) ok = ok && wait(bar(EMPTY + s), (use - 1) & 1, stop, a.status);
        if (!ok) return 0u;
        if (rank == 0) mbar_arrive_expect_tx(bar(FULL + s), 2 * kStage);
        *dst = sbase + kRingOff + s * kStage;
        ++n;
        return full0 + 8 * s;
      };
      for (int x = x0, t = t_first; ok && x < x1; ++t) {
        const int4 tile = plan.tile[t];
        const int begin = plan.cum[t], end = min(x1, plan.cum[t + 1]);
        const int nb = end - x;
        // the last block first: scores that a distance bias shapes fall along the way, and
        // the running maximum seldom rises
        const int row0 = (plan.seq_base[tile.x] + tile.w + (end - 1 - begin)) * kChunkBlk;
        if (nq > 0) ok = wait(bar(QEMPTY), (nq - 1) & 1, stop, a.status);
        if (!ok) break;
        ++nq;
        if (rank == 0) mbar_arrive_expect_tx(bar(QFULL), 2 * kQBytes);
        for (int c = 0; c < 8; ++c)
          tma_load_2d_pair(sbase + c * 16384, &maps.q, 64 * c, tile.y + 128 * rank, qfull);
        for (int i = 0; ok && i <= nb; ++i) {
          if (i < nb) {
            for (int h = 0; ok && h < 2; ++h) {
              uint32_t dst;
              const uint32_t f = stage(&dst);
              if (!ok) break;
              for (int c = 0; c < 4; ++c)
                tma_load_2d_pair(dst + c * 4096, &maps.k, 256 * h + 64 * c, row0 - i * kChunkBlk + 32 * rank, f);
            }
          }
          if (i > 0) {
            for (int h = 0; ok && h < 2; ++h) {
              uint32_t dst;
              const uint32_t f = stage(&dst);
              if (!ok) break;
              // columns 0..255 in halves of 128; 256..447 in halves of 96 (and 32 not read)
              const int col = h == 0 ? 128 * rank : 256 + 96 * rank;
              for (int c = 0; c < 2; ++c)
                tma_load_2d_pair(dst + c * 8192, &maps.v, col + 64 * c, row0 - (i - 1) * kChunkBlk, f);
            }
          }
        }
        x = end;
      }
      if (!ok) {   // copies in flight land within microseconds: 1 ms before shared memory goes
        const long long t0 = clock64();
        while (clock64() - t0 < 2000000) {
        }
      }
    }
  } else if (warp == 5) {
    // ---------------- products ----------------
    // The whole warp walks the schedule, so that stages and addresses stay uniform, and one
    // elected lane issues: with a single thread's loop each product waits for its
    // descriptors to move to uniform registers (87 cycles a product instead of 45 to 64).
    if (rank == 0) {
      constexpr uint32_t kIdQK = idesc_bf16(256, 64, false, false);
      constexpr uint32_t kIdV0 = idesc_bf16(256, 256, false, true);
      constexpr uint32_t kIdV1 = idesc_bf16(256, 192, false, true);
      const uint64_t d0 = smem_desc(sbase, 16, 1024, SWZ_128B), dv = smem_desc(sbase, 8192, 1024, SWZ_128B);
      const uint32_t hi = static_cast<uint32_t>(d0 >> 32);       // the same for every operand
      const uint32_t lq = static_cast<uint32_t>(d0), lk = lq + (kRingOff >> 4), lp = lq + (kPOff >> 4);
      const uint32_t lv = static_cast<uint32_t>(dv) + (kRingOff >> 4);
      uint32_t s = 0, round = 0;                   // next stage, and its use (parity)
      uint32_t nq = 0, ns = 0, np = 0;             // tiles, scores and value products so far
      bool ok = true;
      auto next = [&]() {
        if (++s == kStages) {
          s = 0;
          round ^= 1;
        }
      };
      for (int x = x0, t = t_first; ok && x < x1; ++t) {
        const int end = min(x1, plan.cum[t + 1]);
        const int nb = end - x;
        ok = warp_wait(bar(QFULL), nq & 1, stop, a.status);
        for (int i = 0; ok && i <= nb; ++i) {
          if (i < nb) {
            if (ns > 0) ok = warp_wait(bar(SEMPTY), (ns - 1) & 1, stop, a.status);
            for (int h = 0; ok && h < 2; ++h) {
              ok = warp_wait(bar(FULL + s), round, stop, a.status);
              if (!ok) break;
              tc_fence_after();
              const uint32_t la = lq + ((h * 65536) >> 4), lb = lk + s * (kStage >> 4);
              if (elect_one()) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    mma_f16_ss_pair(tmem + kColS, la + ((c * 16384 + k * 32) >> 4), hi,
                                    lb + ((c * 4096 + k * 32) >> 4), hi, kIdQK, c + k > 0 ? 1u : h);
                mma_commit_pair(bar(EMPTY + s));
                if (h == 1) {
                  mma_commit_pair(bar(SFULL));
                  if (i == nb - 1) mma_commit_pair(bar(QEMPTY));
                }
              }
              __syncwarp();
              next();
            }
            ++ns;
          }
          if (ok && i > 0) {
            ok = warp_wait(bar(PFULL), np & 1, stop, a.status);
            if (ok && i == 1 && nq > 0) ok = warp_wait(bar(OEMPTY), (nq - 1) & 1, stop, a.status);
            for (int h = 0; ok && h < 2; ++h) {
              ok = warp_wait(bar(FULL + s), round, stop, a.status);
              if (!ok) break;
              tc_fence_after();
              const uint32_t lb = lv + s * (kStage >> 4);
              if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma_f16_ss_pair(tmem + 256 * h, lp + ((k * 32) >> 4), hi, lb + ((k * 2048) >> 4), hi,
                                  h == 0 ? kIdV0 : kIdV1, k > 0 ? 1u : (i > 1 ? 1u : 0u));
                mma_commit_pair(bar(EMPTY + s));
                if (h == 1) mma_commit_pair(bar(PV));
              }
              __syncwarp();
              next();
            }
            ++np;
          }
        }
        ++nq;
        x = end;
      }
      if (!ok) {   // let issued products drain before tensor memory is freed
        const long long t0 = clock64();
        while (clock64() - t0 < 2000000) {
        }
      }
    }
  } else {
    // ---------------- softmax and results: thread = row ----------------
    const int r = threadIdx.x;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tS = tmem + kColS + lanes, tO = tmem + lanes;
    const uint32_t sempty = dsmem_addr(bar(SEMPTY), 0), pfull = dsmem_addr(bar(PFULL), 0),
                   oempty = dsmem_addr(bar(OEMPTY), 0);
    uint32_t ns = 0, np = 0;
    bool ok = true;
    for (int x = x0, t = t_first; ok && x < x1; ++t) {
      const int4 tile = plan.tile[t];
      const int begin = plan.cum[t], after = plan.cum[t + 1], end = min(x1, after);
      const int nb = end - x;
      const int base = plan.seq_base[tile.x], blk = tile.w + (end - 1 - begin);     // the first block
      const int row = static_cast<int>(rank) * 128 + r;
      RowState<MODS> st(a, plan, tile, row, row < tile.z);
      for (int i = 0; ok && i < nb; ++i) {
        const ulonglong2 rows = plan.seen[base + blk - i];
        ok = warp_wait(bar(SFULL), ns & 1, stop, a.status);
        ++ns;
        if (!ok) break;
        tc_fence_after();
        float v[64];
        tmem_ld32(tS, v);
        tmem_ld32(tS + 32, v + 32);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(sempty);
        uint32_t p[32];
        const float alpha = st.weights(v, (blk - i) * kChunkBlk, rows, p);
        // the value product before this one is done: P may be written, O rescaled
        if (i > 0) {
          ok = warp_wait(bar(PV), (np - 1) & 1, stop, a.status);
          if (!ok) break;
          tc_fence_after();
          rescale_rows(tO, alpha);
        }
        store_weights(sbase + kPOff, r, p);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && !(warp == 0 && np == static_cast<uint32_t>(a.fault_block))) mbar_arrive_cluster(pfull);
        ++np;
      }
      if (!ok) break;
      ok = warp_wait(bar(PV), (np - 1) & 1, stop, a.status);
      if (!ok) break;
      tc_fence_after();
      store_rows<kPairRows>(a, plan, inverse_sum(st.l, st.lr), lse_of(st.m, st.l), tO, tile,
                                static_cast<int>(rank) * 128 + 32 * warp, begin >= x0 && after <= x1,
                                2 * worker + (begin < x0 ? 0 : 1), sbase + kPOff + warp * 32 * 128);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(oempty);
      x = end;
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive_wait();       // neither CTA's shared or tensor memory goes while the other uses it
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

std::mutex g_mu;

template <bool MODS>
cudaError_t configure(int dev) {
  static bool done[64] = {};
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_mu);
  if (done[dev]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(pair_kernel<MODS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e == cudaSuccess) done[dev] = true;
  return e;
}

template <bool MODS>
cudaError_t launch(const ChunkArgs& a, const ChunkPlan& p, int workers, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = configure<MODS>(dev);
  if (e != cudaSuccess) return e;
  Maps maps;
  std::memset(static_cast<void*>(&maps), 0, sizeof(maps));
  const int64_t kv_rows = (p.cap_blocks + 1) * kChunkBlk;
  e = encode_rows(&maps.q, a.q, static_cast<int64_t>(a.T) * a.H, 128);
  if (e == cudaSuccess) e = encode_rows(&maps.k, p.kv, kv_rows, 32);
  if (e == cudaSuccess) e = encode_rows(&maps.v, p.kv, kv_rows, 64);
  if (e != cudaSuccess) return e;
  return launch_programmatic(pair_kernel<MODS>, dim3(2 * workers), dim3(kThreads), kSmem, stream, a, p, maps);
}

}  // namespace

cudaError_t encode_rows(CUtensorMap* m, const void* base, int64_t rows, int box_rows) {
  const EncodeTiledFn fn = encode_tiled();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dim[2] = {kQkDim, static_cast<cuuint64_t>(rows)};
  const cuuint64_t pitch[1] = {kQkDim * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t step[2] = {1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dim, pitch, box, step,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Pairs that the current device holds at once: asked once a device.
cudaError_t pair_workers(int* workers) {
  static int known[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = configure<false>(dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(g_mu);
  if (known[dev] == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, pair_kernel<false>, &cfg);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorNotSupported;
    known[dev] = n;
  }
  *workers = known[dev];
  return cudaSuccess;
}

cudaError_t launch_chunk_pair(const ChunkArgs& a, const ChunkPlan& p, int workers, cudaStream_t stream) {
  return a.cap > 0.f || a.slopes != nullptr ? launch<true>(a, p, workers, stream)
                                            : launch<false>(a, p, workers, stream);
}

}  // namespace smla
