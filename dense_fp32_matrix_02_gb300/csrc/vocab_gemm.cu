// The products of the vocabulary losses on the 5th-generation tensor cores,
// one kernel whose epilogue makes what the losses need of each 256 × 256
// tile, so that no logits are stored:
//   Stats  z = X·Wᵀ:  per row and 128 columns max and Σ exp, and the logits
//          of the row's targets;
//   Grad   z = X·W_pᵀ: G = g·τ·(exp(z/τ − lse) − q), rounded to 16 bits;
//   Dx     G·W_p, added into fp32 slots (one per split of the depth);
//   Dw     Gᵀ·X, rounded to 16 bits.
//
// Persistent clusters of two CTAs, one pair per two SMs, walk the tiles.  A
// pair works on one tile by tcgen05.mma.cta_group::2 (M 256, N 256, K 16):
// each CTA holds 128 rows of A and 128 columns of B in its shared memory
// (32 KB a k-block of 64), the tensor cores read B from both, and each CTA's
// TMEM receives its 128 rows × 256 columns of the result.  Against a tile of
// 128 × 256 per CTA this loads a third less per multiply (measured with the
// kernels below).  Two accumulators of 256 columns fill TMEM, so a tile's
// epilogue overlaps the next tile's products.
//   warp 0      TMA producer of its own CTA's halves, into a ring; the bytes
//               of both CTAs count on the first CTA's barrier.
//   warp 1      of the first CTA: MMA issuer.  tcgen05.commit releases the
//               stage, and publishes the accumulator, in both CTAs.
//   warps 2-9   epilogue: warp w reads TMEM lanes 32·(w mod 4) + 0..31 (its
//               rows) and one half of the columns.
// Operands lie K-major (X and W in the logits; G in Dx) or along the other
// axis (W in Dx; G and X in Dw), as they are stored: no transposes.
// Every wait is bounded (common.cuh); a CTA that gives up records it, lets
// its copies and products land, and leaves without further stores.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstring>

#include "kernels.h"
#include "tcgen05.cuh"
#include "vocab.cuh"

namespace gemm_f32_impl {
namespace vocab {

constexpr int kBK = 64;
constexpr int kHalf = 128;                   // rows of A, columns of B a CTA
constexpr int kPartBytes = kHalf * kBK * 2;  // 16 KB: one operand, one stage
constexpr int kStageBytes = 2 * kPartBytes;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kStagingBytes = 4096;          // one epilogue warp's block
constexpr int kTmemCols = 512;
constexpr long long kDrainNs = 2000000000LL;
constexpr uint32_t kSleepNs = 100000;
constexpr int kGroup = 16;  // tile rows walked together (L2 reuse)
constexpr float kLog2e = 1.4426950408889634f;

template <int PRODUCT>
struct Shape {
  static constexpr bool kMnA = PRODUCT == kVocabDw;  // A along M
  static constexpr bool kMnB = PRODUCT == kVocabDx || PRODUCT == kVocabDw;
  static constexpr bool kStaged = PRODUCT != kVocabStats;
  static constexpr int kStages = kStaged ? 6 : 7;
  static constexpr int kOffStaging = kStages * kStageBytes;
  static constexpr int kOffCtl =
      kOffStaging + (kStaged ? kEpiWarps * kStagingBytes : 0);
  struct __align__(8) Control {
    uint64_t full[kStages];   // TMA of both CTAs -> MMA (first CTA's is used)
    uint64_t empty[kStages];  // MMA completion -> producers
    uint64_t acc_full[2];     // last MMA of a tile -> epilogues
    uint64_t acc_empty[2];    // epilogue warps of both CTAs -> MMA
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort;
  };
  static constexpr int kSmemBytes = kOffCtl + (int)sizeof(Control) + 1024;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

// ------------------------------------------------ CTA-pair instructions
__device__ __forceinline__ void tmem_alloc2(uint32_t slot, uint32_t ncols) {
  asm volatile(
      "tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
          slot),
      "r"(ncols)
      : "memory");
}

__device__ __forceinline__ void tmem_relinquish2() {
  asm volatile(
      "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::
          : "memory");
}

__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr,
                                              uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(
                   taddr),
               "r"(ncols)
               : "memory");
}

__device__ __forceinline__ void mma2_f16_ss(uint32_t d_tmem, uint64_t a_desc,
                                            uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(
          d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// One arrival on the barrier at this offset of both CTAs of the pair once
// every MMA this thread issued before has completed.
__device__ __forceinline__ void tc_commit2(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
      ".multicast::cluster.b64 [%0], %1;\n" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

// 2-D tile into this CTA's shared memory; the bytes count on `bar`, a
// shared::cluster address that may lie in the pair's other CTA.
__device__ __forceinline__ void tma_load2_2d(uint32_t dst, const void* tmap,
                                             uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx"
      "::bytes.cta_group::2 [%0], [%1, {%3, %4}], [%2];\n" ::"r"(dst),
      "l"(tmap), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile(
      "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(
          bar)
      : "memory");
}

// As mbar_try_wait, acquiring what threads of the other CTA released.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar,
                                                      uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], "
      "%2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity,
                                             long long limit_ns,
                                             volatile int* abort) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if ((i & 15u) == 0) {
      if (abort && *abort) return false;
      if ((long long)(globaltimer_ns() - t0) > limit_ns) return false;
    }
  }
}

// 3-D fp32 store and in-memory addition of a block (c0 innermost).
__device__ __forceinline__ void tma_add_3d(const void* tmap, uint32_t src,
                                           int c0, int c1, int c2) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group "
      "[%0, {%2, %3, %4}], [%1];\n" ::"l"(tmap),
      "r"(src), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// 2^x by the hardware's approximation (relative error about 2^-22; x = -Inf
// gives 0), the exponential of all statistics and gradients here.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

template <int AB_TYPE>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (AB_TYPE == 1) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// What the kernel needs beside the tensor maps.
struct Args {
  int T, D, n;        // n: columns of the piece
  int v0;
  VocabTargets targets;
  float2* stats;
  float* picked;
  const float* lse;
  const float* grad_loss;
  long long grad_stride;
  float tau;
  int add;
  uint16_t* dw;       // direct stores (no tensor map fits dW), else null
  long long lddw;
};

// One tile of the walk: its place and its k-blocks.
struct Unit {
  int tm, tn, split, kb0, kb1;
};

__device__ __forceinline__ Unit unit_of(int u, int tiles_m, int tiles_n,
                                        int nk, int splits) {
  Unit w;
  const int tiles = tiles_m * tiles_n;
  w.split = u / tiles;
  tile_coords<kGroup>(u - w.split * tiles, tiles_m, tiles_n, w.tm, w.tn);
  w.kb0 = (int)((long long)nk * w.split / splits);
  w.kb1 = (int)((long long)nk * (w.split + 1) / splits);
  return w;
}

// A row's entries from column c on: the place of the first with id >= c.
__device__ __forceinline__ int first_entry(const int* ids, int top, int c) {
  int lo = 0, hi = top;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ids[mid] < c)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

template <int AB_TYPE, int PRODUCT>
__global__ void __launch_bounds__(kThreads, 1)
    vocab_gemm_kernel(const __grid_constant__ CUtensorMap map_a,
                      const __grid_constant__ CUtensorMap map_b,
                      const __grid_constant__ CUtensorMap map_xp,
                      const __grid_constant__ CUtensorMap map_c, Args p,
                      WaitCfg wc) {
  using Sh = Shape<PRODUCT>;
  using Control = typename Sh::Control;
  constexpr int kStages = Sh::kStages;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  Control* ctl = reinterpret_cast<Control*>(smem + Sh::kOffCtl);
  volatile int* abort = &ctl->abort;
  auto full = [&](int s) { return smem_u32(&ctl->full[s]); };
  auto empty = [&](int s) { return smem_u32(&ctl->empty[s]); };
  auto acc_full = [&](int b) { return smem_u32(&ctl->acc_full[b]); };
  auto acc_empty = [&](int b) { return smem_u32(&ctl->acc_empty[b]); };
  const uint32_t mma_done = smem_u32(&ctl->mma_done);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), 2 * kEpiWarps);
    }
    mbar_init(mma_done, 1);
    ctl->abort = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&map_a);
    prefetch_tmap(&map_b);
  }
  if (warp == 1) {
    tmem_alloc2(smem_u32(&ctl->tmem_base), kTmemCols);
    tmem_relinquish2();
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();  // the other CTA's barriers are initialised
  tc_fence_after_sync();
  const uint32_t tmem = ctl->tmem_base;
  griddep_wait();  // everything read or written may belong to the kernel before

  const VocabHeader* header = p.targets.header;
  const int learnt = header->learnt;
  const int rows = PRODUCT == kVocabDw ? p.n : learnt;
  const int cols = Sh::kMnB ? p.D : p.n;
  const int depth = PRODUCT == kVocabDw   ? learnt
                    : PRODUCT == kVocabDx ? p.n
                                          : p.D;
  const int splits = PRODUCT == kVocabDx ? header->dx_splits : 1;
  const int tiles_m = (rows + kVocabTile - 1) / kVocabTile;
  const int tiles_n = (cols + kVocabTile - 1) / kVocabTile;
  const int nk = (depth + kBK - 1) / kBK;
  const int units = tiles_m * tiles_n * splits;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const bool packed = header->packed != 0;
      const void* ma = &map_a;
      const void* mb = &map_b;
      if (PRODUCT == kVocabDw) {
        if (packed) mb = &map_xp;
      } else if (PRODUCT != kVocabDx) {
        if (packed) ma = &map_xp;
      }
      int it = 0;
      if (!(wc.debug & kDebugStallProducer)) {
        for (int u = pair; u < units && !*abort; u += pairs) {
          const Unit w = unit_of(u, tiles_m, tiles_n, nk, splits);
          const int m0 = w.tm * kVocabTile + (int)rank * kHalf;
          const int n0 = w.tn * kVocabTile + (int)rank * kHalf;
          for (int kb = w.kb0; kb < w.kb1; ++kb) {
            const int s = it % kStages;
            if (it >= kStages &&
                !bounded_wait(empty(s), ((it / kStages) - 1) & 1, wc.limit,
                              abort, 0)) {
              *abort = 1;
              record_status(wc.status, kStatusTimeoutEmpty);
              break;
            }
            if (rank == 0) mbar_arrive_expect_tx(full(s), 2 * kStageBytes);
            const uint32_t bar = cluster_map(full(s), 0);
            const uint32_t a = sbase + s * kStageBytes, b = a + kPartBytes;
            if (Sh::kMnA) {
              tma_load2_2d(a, ma, bar, m0, kb * kBK);
              tma_load2_2d(a + kPartBytes / 2, ma, bar, m0 + 64, kb * kBK);
            } else {
              tma_load2_2d(a, ma, bar, kb * kBK, m0);
            }
            if (Sh::kMnB) {
              tma_load2_2d(b, mb, bar, n0, kb * kBK);
              tma_load2_2d(b + kPartBytes / 2, mb, bar, n0 + 64, kb * kBK);
            } else {
              tma_load2_2d(b, mb, bar, kb * kBK, n0);
            }
            ++it;
          }
        }
      }
      if (*abort && rank == 0) {  // let the copies still in flight land
        for (int k = it > kStages ? it - kStages : 0; k < it; ++k)
          if (!bounded_wait(full(k % kStages), (k / kStages) & 1, kDrainNs,
                            nullptr, 0))
            record_status(wc.status, kStatusTimeoutDrain);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && rank != 0) {
      // the last arrival from the first CTA's products: nothing of the pair
      // still signals this CTA when it leaves
      if (!wait_cluster(mma_done, 0, 2 * wc.limit + kDrainNs, nullptr))
        record_status(wc.status, kStatusTimeoutDrain);
    }
    if (lane == 0 && rank == 0) {
      const uint32_t idesc =
          idesc_f16(256, 256, AB_TYPE, Sh::kMnB) | (Sh::kMnA ? 1u << 15 : 0u);
      int it = 0;
      bool ok = true;
      for (int u = pair, i = 0; ok && u < units; u += pairs, ++i) {
        const Unit w = unit_of(u, tiles_m, tiles_n, nk, splits);
        const int b = i & 1;
        if (i >= 2 && !wait_cluster(acc_empty(b), ((i >> 1) - 1) & 1,
                                    wc.limit, abort)) {
          *abort = 1;
          record_status(wc.status, kStatusTimeoutMma);
          break;
        }
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem + b * 256;
        for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
          const int s = it % kStages;
          if (!wait_cluster(full(s), (it / kStages) & 1, wc.limit, abort)) {
            *abort = 1;
            record_status(wc.status, kStatusTimeoutFull);
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t a0 = sbase + s * kStageBytes, b0 = a0 + kPartBytes;
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) {
            // 16 k: 32 bytes along a K-major row, 16 rows of 128 bytes else
            const uint64_t ad =
                Sh::kMnA ? smem_desc_sw128(a0 + 2048 * kk, kPartBytes / 2, 1024)
                         : smem_desc_sw128(a0 + 32 * kk, 16, 1024);
            const uint64_t bd =
                Sh::kMnB ? smem_desc_sw128(b0 + 2048 * kk, kPartBytes / 2, 1024)
                         : smem_desc_sw128(b0 + 32 * kk, 16, 1024);
            mma2_f16_ss(d_tmem, ad, bd, idesc, kb != w.kb0 || kk != 0);
          }
          tc_commit2(empty(s));
        }
        if (ok) tc_commit2(acc_full(b));
      }
      // no MMA may still run when TMEM is freed at the end
      tc_commit2(mma_done);
      if (!wait_cluster(mma_done, 0, kDrainNs, nullptr))
        record_status(wc.status, kStatusTimeoutDrain);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;         // TMEM lane quarter
    const int h = (warp - 2) >> 2;  // column half
    const uint32_t lane_bits = (uint32_t)(q * 32) << 16;
    // staging: row (lane) of 128 bytes, its 16-byte chunk j at j ^ (row mod
    // 8), the layout a 128-byte-swizzle TMA store reads
    unsigned char* stg = smem + Sh::kOffStaging + (warp - 2) * kStagingBytes;
    const uint32_t stg_s =
        sbase + Sh::kOffStaging + (warp - 2) * kStagingBytes;
    const float c2 = p.targets.inv_tau * kLog2e;
    const float inv_scale = header->inv_scale;
    const int store_rows = PRODUCT == kVocabGrad ? p.T : rows;
    for (int u = pair, i = 0; u < units; u += pairs, ++i) {
      const Unit w = unit_of(u, tiles_m, tiles_n, nk, splits);
      const int b = i & 1;
      const int m0 = w.tm * kVocabTile + (int)rank * kHalf + q * 32;
      const int r = m0 + lane;
      const int n0 = w.tn * kVocabTile + h * 128;

      // this row's targets, while the tile accumulates
      const int* ids = nullptr;
      const float* log_q = nullptr;
      int at = 0, next = INT_MAX;  // next: id of the next entry, v0 taken off
      float shift = 0.f, g = 0.f;
      if (PRODUCT == kVocabStats || PRODUCT == kVocabGrad) {
        if (r < learnt) {
          const long long t = p.targets.token[r];
          ids = p.targets.ids + t * p.targets.top;
          at = p.targets.top == 1 ? (ids[0] < p.v0 + n0 ? 1 : 0)
                                  : first_entry(ids, p.targets.top, p.v0 + n0);
          if (at < p.targets.top) next = ids[at] - p.v0;
          if (PRODUCT == kVocabGrad) {
            log_q = p.targets.log_q + t * p.targets.top;
            shift = p.lse[t] * kLog2e;
            g = p.grad_loss[t * p.grad_stride] * p.tau * header->scale;
          }
        }
      }

      const bool ok =
          bounded_wait(acc_full(b), (i >> 1) & 1, wc.limit, abort, kSleepNs);
      if (!__all_sync(0xffffffffu, ok)) {
        *abort = 1;
        if (lane == 0) record_status(wc.status, kStatusTimeoutMma);
        break;
      }
      tc_fence_after_sync();
      float peak = -INFINITY, sum = 0.f;
#pragma unroll 1
      for (int c0 = 0; c0 < 128; c0 += 32) {
        uint32_t v[32];
        tmem_ld32(tmem + lane_bits + b * 256 + h * 128 + c0, v);
        tmem_ld_wait();
        if (c0 == 96) {
          // all of this warp's part of the accumulator is in registers
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(cluster_map(acc_empty(b), 0));
        }
        const int n = n0 + c0;
        if (n >= cols) continue;  // (c0 = 96 is never skipped above)
        float f[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[j]);

        if constexpr (PRODUCT == kVocabStats) {
          while (__any_sync(0xffffffffu, next < n + 32)) {
            if (next < n + 32) {
              float z = 0.f;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (next == n + j) z = f[j];
              p.picked[(long long)r * p.targets.top + at] =
                  z * p.targets.inv_tau;
              ++at;
              next = at < p.targets.top ? ids[at] - p.v0 : INT_MAX;
            }
            __syncwarp();
          }
          if (n + 32 > cols) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (n + j >= cols) f[j] = -INFINITY;
          }
          float top4[4] = {f[0], f[1], f[2], f[3]};
#pragma unroll
          for (int j = 4; j < 32; ++j) top4[j & 3] = fmaxf(top4[j & 3], f[j]);
          const float here = fmaxf(fmaxf(top4[0], top4[1]),
                                   fmaxf(top4[2], top4[3]));
          const float now = fmaxf(peak, here * c2);
          // a stretch of -Inf only: every term is 0, not exp(-Inf + Inf)
          const float ref = now == -INFINITY ? 0.f : now;
          float s4[4] = {sum * exp2_fast(peak - ref), 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 32; ++j)
            s4[j & 3] += exp2_fast(fmaf(f[j], c2, -ref));
          sum = (s4[0] + s4[1]) + (s4[2] + s4[3]);
          peak = now;
        } else {
          if constexpr (PRODUCT == kVocabGrad) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              f[j] = exp2_fast(fmaf(f[j], c2, -shift));
            while (__any_sync(0xffffffffu, next < n + 32)) {
              if (next < n + 32) {
                const float qj = expf(log_q[at]);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (next == n + j) f[j] -= qj;
                ++at;
                next = at < p.targets.top ? ids[at] - p.v0 : INT_MAX;
              }
              __syncwarp();
            }
            // rows past the learnt tokens are zeros: Dw sums over them up
            // to a multiple of 64
#pragma unroll
            for (int j = 0; j < 32; ++j) f[j] = r < learnt ? f[j] * g : 0.f;
          }
          if constexpr (PRODUCT == kVocabDw) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              f[j] = nk > 0 ? f[j] * inv_scale : 0.f;
          }
          if constexpr (PRODUCT == kVocabDx) {
            if (w.kb0 == w.kb1) {
#pragma unroll
              for (int j = 0; j < 32; ++j) f[j] = 0.f;
            }
            // fp32, 32 columns: one staged block
            if (lane == 0) bulk_wait_group_read<0>();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<float4*>(stg + lane * 128 +
                                         ((j ^ (lane & 7)) << 4)) =
                  make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2],
                              f[4 * j + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && m0 < learnt) {
              if (p.add)
                tma_add_3d(&map_c, stg_s, n, m0, w.split);
              else
                tma_store_3d(&map_c, stg_s, n, m0, w.split);
              bulk_commit_group();
            }
          } else if (PRODUCT == kVocabDw && p.dw) {
            if (r < rows) {
              uint16_t* out = p.dw + (long long)r * p.lddw + n;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (n + j < cols)
                  out[j] = (uint16_t)pack16<AB_TYPE>(f[j], 0.f);
            }
          } else {
            // 16-bit, 64 columns: half a staged block at a time
            if ((c0 & 32) == 0) {
              if (lane == 0) bulk_wait_group_read<0>();
              __syncwarp();
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int chunk = (c0 & 32) / 8 + j;
              *reinterpret_cast<uint4*>(stg + lane * 128 +
                                        ((chunk ^ (lane & 7)) << 4)) =
                  make_uint4(pack16<AB_TYPE>(f[8 * j], f[8 * j + 1]),
                             pack16<AB_TYPE>(f[8 * j + 2], f[8 * j + 3]),
                             pack16<AB_TYPE>(f[8 * j + 4], f[8 * j + 5]),
                             pack16<AB_TYPE>(f[8 * j + 6], f[8 * j + 7]));
            }
            // the block is whole, or its other half lies past the columns
            if ((c0 & 32) || n + 32 >= cols) {
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0 && m0 < store_rows) {
                tma_store_2d(&map_c, stg_s, n - (c0 & 32), m0);
                bulk_commit_group();
              }
            }
          }
        }
      }
      if (PRODUCT == kVocabStats && r < learnt && n0 < cols)
        p.stats[(long long)(w.tn * 2 + h) * p.T + r] = make_float2(peak, sum);
    }
    if (Sh::kStaged && lane == 0) bulk_wait_group<0>();
  }

  griddep_launch_dependents();
  tc_fence_before_sync();
  __syncwarp();  // reconverge the warps whose roles ran on one lane
  __syncthreads();
  cluster_sync_all();  // the pair's products and copies are over
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc2(tmem, kTmemCols);
  }
}

// A row-major 16-bit matrix (x contiguous), 64 × by boxes, 128-byte swizzle.
bool encode_16(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* m,
               int type, const void* base, long long x, long long y,
               long long ld, int by) {
  const cuuint64_t dims[2] = {(cuuint64_t)x, (cuuint64_t)y};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)by};
  const cuuint32_t estr[2] = {1, 1};
  return encode(m,
                type == GEMM_F32_MIXED_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                            : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                2, const_cast<void*>(base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int AB_TYPE, int PRODUCT>
cudaError_t launch(const VocabGemm& p, int sm_count, const WaitCfg& wc,
                   cudaStream_t stream) {
  using Sh = Shape<PRODUCT>;
  auto encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  CUtensorMap a, b, xp, c;
  std::memset(&c, 0, sizeof(c));
  Args k = {};
  k.T = p.T;
  k.D = p.D;
  k.n = p.n;
  k.v0 = p.v0;
  k.targets = p.targets;
  k.stats = p.stats;
  k.picked = p.picked;
  k.lse = p.lse;
  k.grad_loss = p.grad_loss;
  k.grad_stride = p.grad_stride;
  k.tau = p.tau;
  k.add = p.add;
  bool ok = true;
  // X as given may have no tensor map (its alignment): then only the packed
  // copy is read
  const bool x_fits = (reinterpret_cast<uintptr_t>(p.X) & 15u) == 0 &&
                      p.ldx % 8 == 0;
  auto encode_x = [&](CUtensorMap* as_given, int by) {
    ok = ok && encode_16(encode, &xp, p.type, p.Xp, p.D, p.rows_xp, p.ldxp, by);
    if (x_fits)
      ok = ok && encode_16(encode, as_given, p.type, p.X, p.D, p.T, p.ldx, by);
    else
      *as_given = xp;
  };
  if (PRODUCT == kVocabStats || PRODUCT == kVocabGrad) {
    encode_x(&a, kHalf);
    ok = ok && encode_16(encode, &b, p.type, p.W, p.D, p.n, p.ldw, kHalf);
    if (PRODUCT == kVocabGrad)
      ok = ok && encode_16(encode, &c, p.type, p.G, p.n, p.T, p.ldg, 32);
  } else if (PRODUCT == kVocabDx) {
    ok = ok && encode_16(encode, &a, p.type, p.G, p.n, p.T, p.ldg, kHalf) &&
         encode_16(encode, &b, p.type, p.W, p.D, p.n, p.ldw, kBK);
    xp = a;
    const cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)p.T,
                                (cuuint64_t)p.max_splits};
    const cuuint64_t strides[2] = {(cuuint64_t)p.ld_slot * 4,
                                   (cuuint64_t)p.ld_slot * 4 * p.T};
    const cuuint32_t box[3] = {32, 32, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    ok = ok &&
         encode(&c, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, p.slots, dims, strides,
                box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  } else {
    ok = ok && encode_16(encode, &a, p.type, p.G, p.n, p.T, p.ldg, kBK);
    encode_x(&b, kBK);
    if ((reinterpret_cast<uintptr_t>(p.dW) & 15u) == 0 && p.lddw % 8 == 0) {
      ok = ok && encode_16(encode, &c, p.type, p.dW, p.D, p.n, p.lddw, 32);
    } else {
      k.dw = static_cast<uint16_t*>(p.dW);
      k.lddw = p.lddw;
    }
  }
  if (!ok) return cudaErrorInvalidValue;
  auto fn = vocab_gemm_kernel<AB_TYPE, PRODUCT>;
  cudaError_t e =
      ensure_smem_attr(reinterpret_cast<const void*>(fn), Sh::kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(fn, dim3(2 * (sm_count / 2)), dim3(kThreads),
                            Sh::kSmemBytes, stream, 2, a, b, xp, c, k, wc);
}

template <int PRODUCT>
cudaError_t launch_typed(const VocabGemm& p, int sm_count, const WaitCfg& wc,
                         cudaStream_t stream) {
  return p.type == GEMM_F32_MIXED_BF16
             ? launch<1, PRODUCT>(p, sm_count, wc, stream)
             : launch<0, PRODUCT>(p, sm_count, wc, stream);
}

}  // namespace vocab

cudaError_t launch_vocab_gemm(VocabProduct product, const VocabGemm& p,
                              int sm_count, const WaitCfg& wc,
                              cudaStream_t stream) {
  switch (product) {
    case kVocabStats:
      return vocab::launch_typed<kVocabStats>(p, sm_count, wc, stream);
    case kVocabGrad:
      return vocab::launch_typed<kVocabGrad>(p, sm_count, wc, stream);
    case kVocabDx:
      return vocab::launch_typed<kVocabDx>(p, sm_count, wc, stream);
    default:
      return vocab::launch_typed<kVocabDw>(p, sm_count, wc, stream);
  }
}

}  // namespace gemm_f32_impl
