// Vocabulary losses: softmax cross entropy and distillation of z = X·Wᵀ,
// forward and backward (the definitions are in include/gemm_f32.h).
//
// Both losses are one computation.  Token t has a sparse target distribution
// q_t (one entry for cross entropy, the teacher's softmax over its entries
// for distillation) and, with p_t = softmax(z_t/τ),
//   loss_t = τ²·Σ_j q_tj·(log q_tj − (z[t][id_tj]/τ − lse_t)),
//   dL/dz_t = g_t·τ·(p_t − q_t)
// (cross entropy: q = 1, τ = 1).  A call runs
//   1. the targets: entries sorted by id with log q; the tokens that are
//      learnt from, numbered (everything after works on those rows only);
//   2. forward: the logits piece by piece, each reduced to per-row softmax
//      statistics and the targets' logits; then loss and lse;
//      backward: each piece made again, turned into G = dL/dz, and
//      multiplied by W (dX, added up over the pieces) and by X (dW's rows
//      of that piece).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "gemm_f32.h"
#include "kernels.h"
#include "vocab.cuh"

namespace gemm_f32_impl {
namespace {

// ------------------------------------------------------------- targets
// Distillation: one warp per token.  log q over the entries that count,
// which are ranked by (id, place) and written in that order.
constexpr int kTargetWarps = 4;

__global__ void __launch_bounds__(32 * kTargetWarps)
    distill_targets_kernel(int T, int V, int top,
                           const float* __restrict__ logits, long long ldt,
                           const int64_t* __restrict__ top_ids, long long ldi,
                           float inv_tau, int* __restrict__ ids,
                           float* __restrict__ log_q,
                           uint8_t* __restrict__ flags) {
  __shared__ int s_id[kTargetWarps][kVocabMaxTop];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kTargetWarps + warp;
  if (t >= T) return;
  int* sid = s_id[warp];
  constexpr int kPer = kVocabMaxTop / 32;
  float u[kPer];
  float peak = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int j = lane + 32 * i;
    u[i] = -INFINITY;
    if (j < top) {
      const float l = logits[t * ldt + j];
      const int64_t id = top_ids[t * ldi + j];
      const bool counts = id >= 0 && id < V && l != -INFINITY;
      sid[j] = counts ? (int)id : INT_MAX;
      if (counts) u[i] = l * inv_tau;
      peak = fmaxf(peak, u[i]);
    }
  }
  for (int o = 16; o; o >>= 1)
    peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, o));
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i)  // u = -Inf (no entry) adds nothing
    if (u[i] != -INFINITY) sum += expf(u[i] - peak);
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float log_sum = logf(sum);
  // sum is 0 only where nothing counts (the largest term is 1, or NaN)
  if (lane == 0) flags[t] = sum != 0.f;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int j = lane + 32 * i;
    if (j < top) {
      const int id = sid[j];
      int rank = 0;
      for (int k = 0; k < top; ++k)
        rank += sid[k] < id || (sid[k] == id && k < j);
      ids[(long long)t * top + rank] = id;
      log_q[(long long)t * top + rank] =
          id == INT_MAX ? -INFINITY : (u[i] - peak) - log_sum;
    }
  }
}

// Numbers the tokens that are learnt from, in order, and packs their rows of
// X where they are not read in place (some token is not learnt from, or X
// has no tensor map).  Every block numbers all tokens, 256 a warp at a time
// (the flags come from L2; at 8192 tokens this took a single block followed
// by a packing kernel 17 + 11 us), and writes what belongs to its own share
// of them.  Forward: loss and lse of the other tokens are 0.  Gradients: the
// power of two that brings the largest |g·τ| near 2^14 (binary16 G; 1 for
// bfloat16, whose exponents need no help), and dX's slots.
struct NumberArgs {
  int T, V;
  const int64_t* targets;  // cross entropy
  const uint8_t* flags;    // distillation
  float *loss, *lse;       // forward, else null
  const float* grad_loss;  // gradients, else null
  long long grad_stride;
  float tau;
  int scaled;       // binary16
  int always_pack;  // X has no tensor map
  const uint16_t* X;
  long long ldx;
  uint16_t* Xp;
  long long ldxp;
  int D, piece, pairs, max_splits;
  int share;        // tokens of a block
};

// 16-bit row of n elements, then zeros up to a multiple of 8, to a 16-byte
// aligned row; by one warp.  vec: the source is aligned too.
__device__ __forceinline__ void pack_row(const uint16_t* __restrict__ src,
                                         int n, uint16_t* __restrict__ dst,
                                         bool vec, int lane) {
  for (int c = 8 * lane; c < n; c += 256) {
    uint4 v;
    if (vec && c + 8 <= n) {
      v = *reinterpret_cast<const uint4*>(src + c);
    } else {
      uint32_t e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = c + j < n ? src[c + j] : 0;
      v = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16,
                     e[6] | e[7] << 16);
    }
    *reinterpret_cast<uint4*>(dst + c) = v;
  }
}

__global__ void __launch_bounds__(1024)
    number_tokens_kernel(NumberArgs a, int* __restrict__ ids,
                         float* __restrict__ log_q, int* __restrict__ token,
                         int* __restrict__ row, VocabHeader* header) {
  __shared__ int s_count[32];
  __shared__ float s_max[32];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long own0 = (long long)blockIdx.x * a.share;
  const long long own1 = min((long long)a.T, own0 + a.share);
  int base = 0;
  for (long long t0 = 0; t0 < a.T; t0 += 8192) {
    unsigned votes[8];
    int count = 0;
    int64_t y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const long long t = t0 + warp * 256 + i * 32 + lane;
      y[i] = -1;
      if (t < a.T) y[i] = a.targets ? a.targets[t] : (int64_t)a.flags[t] - 1;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      votes[i] = __ballot_sync(0xffffffffu, y[i] >= 0 && y[i] < a.V);
      count += __popc(votes[i]);
    }
    if (lane == 0) s_count[warp] = count;
    __syncthreads();
    int incl = s_count[lane];
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    int r0 = base + (warp ? __shfl_sync(0xffffffffu, incl, (warp - 1) & 31) : 0);
    base += __shfl_sync(0xffffffffu, incl, 31);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const long long t = t0 + warp * 256 + i * 32 + lane;
      const bool learnt = (votes[i] >> lane) & 1u;
      const int r = r0 + __popc(votes[i] & ((1u << lane) - 1u));
      if (t >= own0 && t < own1) {
        row[t] = learnt ? r : -1;
        if (learnt) token[r] = (int)t;
        if (a.targets) {
          ids[t] = learnt ? (int)y[i] : INT_MAX;
          log_q[t] = learnt ? 0.f : -INFINITY;
        }
        if (a.loss && !learnt) {
          a.loss[t] = 0.f;
          a.lse[t] = 0.f;
        }
      }
      r0 += __popc(votes[i]);
    }
    __syncthreads();
  }
  const bool packed = a.always_pack || base != a.T;
  if (packed) {
    const bool vec = (reinterpret_cast<uintptr_t>(a.X) & 15u) == 0 &&
                     a.ldx % 8 == 0;
    for (long long t = own0 + warp; t < own1; t += 32) {
      const int r = row[t];  // written by this block, before the barrier
      if (r >= 0)
        pack_row(a.X + t * a.ldx, a.D, a.Xp + r * a.ldxp, vec, lane);
    }
  }
  if (blockIdx.x != 0) return;
  if (packed) {  // Dw sums over the rows up to a multiple of 64
    for (int r = base + warp; r < (base + 63) / 64 * 64; r += 32)
      for (int c = 8 * lane; c < a.D; c += 256)
        *reinterpret_cast<uint4*>(a.Xp + r * a.ldxp + c) =
            make_uint4(0, 0, 0, 0);
  }
  float most = 0.f;
  if (a.grad_loss && a.scaled)
    for (long long t = threadIdx.x; t < a.T; t += 1024) {
      const bool learnt = a.targets
                              ? a.targets[t] >= 0 && a.targets[t] < a.V
                              : a.flags[t] != 0;
      if (learnt) most = fmaxf(most, fabsf(a.grad_loss[t * a.grad_stride]));
    }
  for (int o = 16; o; o >>= 1)
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (lane == 0) s_max[warp] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 32; ++w) most = fmaxf(most, s_max[w]);
    most *= a.tau;
    int e = 0;
    // 0, Inf and NaN: no scale
    if (a.scaled && most > 0.f && most < INFINITY)
      e = min(max(14 - ilogbf(most), -100), 100);
    header->learnt = base;
    header->packed = packed;
    header->dx_splits = a.grad_loss ? vocab_dx_splits(base, a.D, a.piece,
                                                      a.pairs, a.max_splits)
                                    : 1;
    header->scale = ldexpf(1.f, e);
    header->inv_scale = ldexpf(1.f, -e);
  }
}

// W's rows where they have no tensor map, one warp a row.
__global__ void __launch_bounds__(256)
    pack_rows_kernel(const uint16_t* __restrict__ src, long long lds, int cols,
                     uint16_t* __restrict__ dst, long long ldd, int rows) {
  griddep_wait();
  griddep_launch_dependents();
  const int warps = gridDim.x * 8;
  for (long long r = blockIdx.x * 8 + (threadIdx.x >> 5); r < rows; r += warps)
    pack_row(src + r * lds, cols, dst + r * ldd, false, threadIdx.x & 31);
}

// ------------------------------------------------------------- results
__device__ __forceinline__ float2 merge_stats(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  const float ref = m == -INFINITY ? 0.f : m;
  return make_float2(m, a.y * exp2f(a.x - ref) + b.y * exp2f(b.x - ref));
}

// loss and lse of the learnt tokens: 8 rows a block, 128 threads a row that
// share out its statistics (parts of them, [part][T]) and join them in a
// fixed order.
__global__ void __launch_bounds__(1024)
    finish_loss_kernel(VocabTargets tg, int T, int parts,
                       const float2* __restrict__ stats,
                       const float* __restrict__ picked, float tau,
                       float* __restrict__ loss, float* __restrict__ lse) {
  __shared__ float2 s_part[32][8];
  griddep_wait();
  griddep_launch_dependents();
  const int r = blockIdx.x * 8 + (threadIdx.x & 7);
  const int slice = threadIdx.x >> 3, warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const bool here = r < tg.header->learnt;
  // the first warp's later loads, ahead of the statistics'
  long long t = 0;
  int id = INT_MAX;
  float lq = 0.f, at = 0.f;
  if (warp == 0 && here) {
    t = tg.token[r];
    if (lane >> 3 < tg.top) {
      id = tg.ids[t * tg.top + (lane >> 3)];
      lq = tg.log_q[t * tg.top + (lane >> 3)];
      at = picked[(long long)r * tg.top + (lane >> 3)];
    }
  }
  float2 st = make_float2(-INFINITY, 0.f);
  if (here) {
#pragma unroll 4
    for (int e = slice; e < parts; e += 128)
      st = merge_stats(st, stats[(long long)e * T + r]);
  }
  for (int o = 8; o < 32; o <<= 1)
    st = merge_stats(st, make_float2(__shfl_xor_sync(0xffffffffu, st.x, o),
                                     __shfl_xor_sync(0xffffffffu, st.y, o)));
  if (lane < 8) s_part[warp][lane] = st;
  __syncthreads();
  if (warp > 0) return;
  st = make_float2(-INFINITY, 0.f);
  for (int w = lane >> 3; w < 32; w += 4)
    st = merge_stats(st, s_part[w][lane & 7]);
  for (int o = 8; o < 32; o <<= 1)
    st = merge_stats(st, make_float2(__shfl_xor_sync(0xffffffffu, st.x, o),
                                     __shfl_xor_sync(0xffffffffu, st.y, o)));
  const float l = st.x * 0.69314718f + logf(st.y);
  float sum = 0.f;
  for (int j = lane >> 3; id != INT_MAX;) {
    sum += expf(lq) * (lq - (at - l));
    j += 4;
    if (j >= tg.top) break;
    id = tg.ids[t * tg.top + j];
    lq = tg.log_q[t * tg.top + j];
    at = picked[(long long)r * tg.top + j];
  }
  for (int o = 8; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (here && lane < 8) {
    loss[t] = tau * tau * sum;
    lse[t] = l;
  }
}

// dX row by row: the slots' sum in order, rounded; zeros for the tokens that
// are not learnt from.  vec: four columns at a time (dX's rows are 8-byte
// aligned).
template <typename T16>
__global__ void __launch_bounds__(256)
    finish_dx_kernel(int T, int D, const int* __restrict__ row,
                     const VocabHeader* header,
                     const float* __restrict__ slots, long long ld_slot,
                     T16* __restrict__ dX, long long lddx, int vec) {
  griddep_wait();
  griddep_launch_dependents();
  const long long t = blockIdx.x;
  const int r = row[t], splits = header->dx_splits;
  const float inv_scale = header->inv_scale;
  const float* from = slots + (long long)r * ld_slot;
  for (int i = 4 * threadIdx.x; i < D; i += 1024) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r >= 0) {
      for (int s = 0; s < splits; ++s) {
        const float4 a = *reinterpret_cast<const float4*>(
            from + (long long)s * T * ld_slot + i);
        v.x += a.x;
        v.y += a.y;
        v.z += a.z;
        v.w += a.w;
      }
    }
    T16 o[4];
    store16(o, v.x * inv_scale);
    store16(o + 1, v.y * inv_scale);
    store16(o + 2, v.z * inv_scale);
    store16(o + 3, v.w * inv_scale);
    T16* to = dX + t * lddx + i;
    if (vec && i + 4 <= D) {
      *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(o);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < D) to[j] = o[j];
    }
  }
}

// ------------------------------------------------------------- host side
struct VocabCall {
  int type;
  int64_t T, V, D;
  const void* X;
  int64_t ldx;
  const void* W;
  int64_t ldw;
  const int64_t* targets;  // cross entropy
  int64_t top;
  const float* top_logits;  // distillation
  int64_t ldt;
  const int64_t* top_ids;
  int64_t ldi;
  float tau;
  float* loss;  // forward
  float* lse;
  const float* lse_in;  // gradients
  const float* grad_loss;
  int64_t grad_stride;
  void* dX;
  int64_t lddx;
  void* dW;
  int64_t lddw;
  void* ws;
  int64_t ws_bytes;
  cudaStream_t stream;
};

int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Where a call's state lies in its workspace, and the pieces of the
// vocabulary the gradients go through.
struct VocabLayout {
  int64_t piece;       // columns of G
  int64_t max_splits;  // slots of dX
  int64_t ld_pack;     // row stride of the packed copies
  int64_t header, token, row, flags, ids, log_q, x_pack, w_pack, total;
  int64_t stats, picked;  // forward
  int64_t g, slots;       // gradients
};

VocabLayout layout(int64_t T, int64_t V, int64_t D, int64_t top, bool grad,
                   bool pack_w) {
  constexpr int64_t kMostG = 256ll << 20, kMostSlots = 512ll << 20;
  VocabLayout l = {};
  const int64_t rows = std::max<int64_t>(T, 1);
  l.ld_pack = up(D, 8);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += up(bytes, 256);
    return here;
  };
  l.header = take(sizeof(VocabHeader));
  l.token = take(rows * 4);
  l.row = take(rows * 4);
  l.flags = take(rows);
  l.ids = take(rows * top * 4);
  l.log_q = take(rows * top * 4);
  l.x_pack = take(up(rows, 64) * l.ld_pack * 2);
  if (pack_w) l.w_pack = take(V * l.ld_pack * 2);
  if (grad) {
    // equal pieces, whole tiles, of at most kMostG bytes of G
    const int64_t widest = std::max<int64_t>(
        kVocabTile, kMostG / (2 * rows) / kVocabTile * kVocabTile);
    const int64_t pieces = (V + widest - 1) / widest;
    l.piece = up((V + pieces - 1) / pieces, kVocabTile);
    const int64_t slot = rows * up(D, 4) * 4;
    l.max_splits = std::min<int64_t>(
        64, std::max<int64_t>(1, kMostSlots / slot));
    l.g = take(rows * l.piece * 2);
    l.slots = take(l.max_splits * slot);
  } else {
    l.stats = take((V + 127) / 128 * rows * 8);
    l.picked = take(rows * top * 4);
  }
  l.total = at;
  return l;
}

bool fits_tensor_map(const void* p, int64_t ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0;
}

int check_call(const VocabCall& c, bool grad, bool distill) {
  if (c.type != GEMM_F32_MIXED_BF16 && c.type != GEMM_F32_MIXED_F16)
    return GEMM_F32_ERR_INVALID_ARG;
  if (c.T < 0 || c.V < 1 || c.D < 1 || c.ldx < c.D || c.ldw < c.D)
    return GEMM_F32_ERR_INVALID_ARG;
  if (c.top < 1 || c.top > kVocabMaxTop) return GEMM_F32_ERR_INVALID_ARG;
  if (!(c.tau > 0.f) || !std::isfinite(c.tau) || !std::isfinite(1.f / c.tau))
    return GEMM_F32_ERR_INVALID_ARG;
  if (distill && (c.ldt < c.top || c.ldi < c.top))
    return GEMM_F32_ERR_INVALID_ARG;
  if (c.ws_bytes < 0) return GEMM_F32_ERR_INVALID_ARG;
  if (!c.W || (grad && !c.dW)) return GEMM_F32_ERR_INVALID_ARG;
  if (grad && (c.lddx < c.D || c.lddw < c.D || c.grad_stride < 0))
    return GEMM_F32_ERR_INVALID_ARG;
  if (c.T > 0) {
    if (!c.X) return GEMM_F32_ERR_INVALID_ARG;
    if (distill ? (!c.top_logits || !c.top_ids) : !c.targets)
      return GEMM_F32_ERR_INVALID_ARG;
    if (grad ? (!c.lse_in || !c.grad_loss || !c.dX) : (!c.loss || !c.lse))
      return GEMM_F32_ERR_INVALID_ARG;
  }
  if (c.T > 0x7fffffff || c.V > 0x7fffffff || c.D > 0x7fffffff)
    return GEMM_F32_ERR_UNSUPPORTED;
  return GEMM_F32_OK;
}

cudaError_t run_checked(const VocabCall& c, bool grad, int sms,
                        const WaitCfg& wc) {
  const int T = (int)c.T, V = (int)c.V, D = (int)c.D, top = (int)c.top;
  cudaStream_t s = c.stream;
  if (T == 0)  // gradients: dW = 0
    return cudaMemset2DAsync(c.dW, c.lddw * 2, 0, c.D * 2, c.V, s);
  const bool w_fits = fits_tensor_map(c.W, c.ldw);
  const bool x_fits = fits_tensor_map(c.X, c.ldx);
  const VocabLayout l = layout(c.T, c.V, c.D, c.top, grad, !w_fits);
  char* ws = static_cast<char*>(c.ws);
  auto* header = reinterpret_cast<VocabHeader*>(ws + l.header);
  int* token = reinterpret_cast<int*>(ws + l.token);
  int* row = reinterpret_cast<int*>(ws + l.row);
  int* ids = reinterpret_cast<int*>(ws + l.ids);
  float* log_q = reinterpret_cast<float*>(ws + l.log_q);
  const float inv_tau = 1.f / c.tau;
  cudaError_t e;

  auto* flags = reinterpret_cast<uint8_t*>(ws + l.flags);
  if (!c.targets) {
    e = launch_pdl(distill_targets_kernel,
                   dim3((T + kTargetWarps - 1) / kTargetWarps),
                   dim3(32 * kTargetWarps), 0, s, T, V, top, c.top_logits,
                   (long long)c.ldt, c.top_ids, (long long)c.ldi, inv_tau,
                   ids, log_q, flags);
    if (e != cudaSuccess) return e;
  }
  NumberArgs na = {};
  na.T = T, na.V = V;
  na.targets = c.targets, na.flags = flags;
  na.loss = c.loss, na.lse = c.lse;
  na.grad_loss = c.grad_loss, na.grad_stride = c.grad_stride;
  na.tau = c.tau;
  na.scaled = c.type == GEMM_F32_MIXED_F16;
  na.always_pack = !x_fits;
  na.X = static_cast<const uint16_t*>(c.X), na.ldx = c.ldx;
  na.Xp = reinterpret_cast<uint16_t*>(ws + l.x_pack), na.ldxp = l.ld_pack;
  na.D = D, na.piece = (int)std::min(l.piece, c.V);
  na.pairs = std::max(1, sms / 2), na.max_splits = (int)l.max_splits;
  const int blocks = std::min(sms, (T + 31) / 32);
  na.share = (T + blocks - 1) / blocks;
  e = launch_pdl(number_tokens_kernel, dim3(blocks), dim3(1024), 0, s, na, ids,
                 log_q, token, row, header);
  if (e != cudaSuccess) return e;
  if (!w_fits) {
    e = launch_pdl(pack_rows_kernel, dim3(std::min(8 * sms, (V + 7) / 8)),
                   dim3(256), 0, s, static_cast<const uint16_t*>(c.W),
                   (long long)c.ldw, D,
                   reinterpret_cast<uint16_t*>(ws + l.w_pack),
                   (long long)l.ld_pack, V);
    if (e != cudaSuccess) return e;
  }
  const char* W = w_fits ? static_cast<const char*>(c.W) : ws + l.w_pack;
  const int64_t ldw = w_fits ? c.ldw : l.ld_pack;

  VocabGemm p = {};
  p.type = c.type;
  p.T = T, p.D = D;
  p.X = c.X, p.ldx = c.ldx;
  p.Xp = ws + l.x_pack, p.ldxp = l.ld_pack, p.rows_xp = (int)up(c.T, 64);
  p.W = W, p.ldw = ldw;
  p.v0 = 0, p.n = V;
  p.targets = VocabTargets{header, token, ids, log_q, top, inv_tau};
  if (!grad) {
    p.stats = reinterpret_cast<float2*>(ws + l.stats);
    p.picked = reinterpret_cast<float*>(ws + l.picked);
    if ((e = launch_vocab_gemm(kVocabStats, p, sms, wc, s)) != cudaSuccess)
      return e;
    return launch_pdl(finish_loss_kernel, dim3((T + 7) / 8), dim3(1024), 0, s,
                      p.targets, T, (V + 127) / 128, p.stats, p.picked, c.tau,
                      c.loss, c.lse);
  }
  p.G = ws + l.g, p.ldg = l.piece;
  p.lse = c.lse_in;
  p.grad_loss = c.grad_loss, p.grad_stride = c.grad_stride, p.tau = c.tau;
  p.slots = reinterpret_cast<float*>(ws + l.slots);
  p.ld_slot = up(c.D, 4), p.max_splits = (int)l.max_splits;
  p.lddw = c.lddw;
  for (int64_t v0 = 0; v0 < c.V; v0 += l.piece) {
    p.v0 = (int)v0, p.n = (int)std::min(l.piece, c.V - v0);
    p.W = W + v0 * ldw * 2;
    p.dW = static_cast<char*>(c.dW) + v0 * c.lddw * 2;
    p.add = v0 > 0;
    for (VocabProduct product : {kVocabGrad, kVocabDx, kVocabDw})
      if ((e = launch_vocab_gemm(product, p, sms, wc, s)) != cudaSuccess)
        return e;
  }
  const int vec = (reinterpret_cast<uintptr_t>(c.dX) & 7u) == 0 &&
                  c.lddx % 4 == 0;
  auto finish = [&](auto* dX) {
    return launch_pdl(
        finish_dx_kernel<std::remove_pointer_t<decltype(dX)>>, dim3(T),
        dim3(256), 0, s, T, D, row, header, p.slots, p.ld_slot, dX,
        (long long)c.lddx, vec);
  };
  return c.type == GEMM_F32_MIXED_BF16
             ? finish(static_cast<__nv_bfloat16*>(c.dX))
             : finish(static_cast<__half*>(c.dX));
}

int run_vocab(const VocabCall& c, bool grad, bool distill) {
  int st = check_call(c, grad, distill);
  if (st != GEMM_F32_OK) return st;
  if (c.T == 0 && !grad) return GEMM_F32_OK;
  const VocabLayout l = layout(c.T, c.V, c.D, c.top, grad,
                               !fits_tensor_map(c.W, c.ldw));
  if (!c.ws || (reinterpret_cast<uintptr_t>(c.ws) & 15u) != 0 ||
      c.ws_bytes < l.total)
    return GEMM_F32_ERR_INVALID_ARG;
  int sms = 0, cc = 0;
  WaitCfg wc;
  cudaError_t e = device_facts(&sms, &cc, &wc);
  if (e != cudaSuccess) return record_cuda_error(e);
  if (cc != 10) return GEMM_F32_ERR_UNSUPPORTED;
  e = run_checked(c, grad, sms, wc);
  return e == cudaSuccess ? GEMM_F32_OK : record_cuda_error(e);
}

}  // namespace
}  // namespace gemm_f32_impl

using namespace gemm_f32_impl;

extern "C" {

int gemm_f32_vocab_ce(int type, int64_t T, int64_t V, int64_t D,
                      const void* X, int64_t ldx, const void* W, int64_t ldw,
                      const int64_t* targets, float* loss, float* lse,
                      void* workspace, int64_t workspace_bytes,
                      gemm_f32_stream_t stream) {
  VocabCall c = {};
  c.type = type, c.T = T, c.V = V, c.D = D;
  c.X = X, c.ldx = ldx, c.W = W, c.ldw = ldw;
  c.targets = targets, c.top = 1, c.tau = 1.f;
  c.loss = loss, c.lse = lse;
  c.ws = workspace, c.ws_bytes = workspace_bytes;
  c.stream = reinterpret_cast<cudaStream_t>(stream);
  return run_vocab(c, false, false);
}

int gemm_f32_vocab_ce_grad(int type, int64_t T, int64_t V, int64_t D,
                           const void* X, int64_t ldx, const void* W,
                           int64_t ldw, const int64_t* targets,
                           const float* lse, const float* grad_loss,
                           int64_t grad_stride, void* dX, int64_t lddx,
                           void* dW, int64_t lddw, void* workspace,
                           int64_t workspace_bytes,
                           gemm_f32_stream_t stream) {
  VocabCall c = {};
  c.type = type, c.T = T, c.V = V, c.D = D;
  c.X = X, c.ldx = ldx, c.W = W, c.ldw = ldw;
  c.targets = targets, c.top = 1, c.tau = 1.f;
  c.lse_in = lse, c.grad_loss = grad_loss, c.grad_stride = grad_stride;
  c.dX = dX, c.lddx = lddx, c.dW = dW, c.lddw = lddw;
  c.ws = workspace, c.ws_bytes = workspace_bytes;
  c.stream = reinterpret_cast<cudaStream_t>(stream);
  return run_vocab(c, true, false);
}

int gemm_f32_vocab_distill(int type, int64_t T, int64_t V, int64_t D,
                           const void* X, int64_t ldx, const void* W,
                           int64_t ldw, int64_t top, const float* top_logits,
                           int64_t ldt, const int64_t* top_ids, int64_t ldi,
                           float temperature, float* loss, float* lse,
                           void* workspace, int64_t workspace_bytes,
                           gemm_f32_stream_t stream) {
  VocabCall c = {};
  c.type = type, c.T = T, c.V = V, c.D = D;
  c.X = X, c.ldx = ldx, c.W = W, c.ldw = ldw;
  c.top = top, c.top_logits = top_logits, c.ldt = ldt;
  c.top_ids = top_ids, c.ldi = ldi, c.tau = temperature;
  c.loss = loss, c.lse = lse;
  c.ws = workspace, c.ws_bytes = workspace_bytes;
  c.stream = reinterpret_cast<cudaStream_t>(stream);
  return run_vocab(c, false, true);
}

int gemm_f32_vocab_distill_grad(
    int type, int64_t T, int64_t V, int64_t D, const void* X, int64_t ldx,
    const void* W, int64_t ldw, int64_t top, const float* top_logits,
    int64_t ldt, const int64_t* top_ids, int64_t ldi, float temperature,
    const float* lse, const float* grad_loss, int64_t grad_stride, void* dX,
    int64_t lddx, void* dW, int64_t lddw, void* workspace,
    int64_t workspace_bytes, gemm_f32_stream_t stream) {
  VocabCall c = {};
  c.type = type, c.T = T, c.V = V, c.D = D;
  c.X = X, c.ldx = ldx, c.W = W, c.ldw = ldw;
  c.top = top, c.top_logits = top_logits, c.ldt = ldt;
  c.top_ids = top_ids, c.ldi = ldi, c.tau = temperature;
  c.lse_in = lse, c.grad_loss = grad_loss, c.grad_stride = grad_stride;
  c.dX = dX, c.lddx = lddx, c.dW = dW, c.lddw = lddw;
  c.ws = workspace, c.ws_bytes = workspace_bytes;
  c.stream = reinterpret_cast<cudaStream_t>(stream);
  return run_vocab(c, true, true);
}

int64_t gemm_f32_vocab_workspace_size(int64_t T, int64_t V, int64_t D,
                                      int64_t top, int grad, int aligned) {
  if (T < 0 || V < 1 || D < 1 || top < 1 || top > kVocabMaxTop ||
      (grad != 0 && grad != 1) || (aligned != 0 && aligned != 1))
    return -GEMM_F32_ERR_INVALID_ARG;
  if (T > 0x7fffffff || V > 0x7fffffff || D > 0x7fffffff)
    return -GEMM_F32_ERR_UNSUPPORTED;
  return layout(T, V, D, top, grad != 0, aligned == 0).total;
}

}  // extern "C"
