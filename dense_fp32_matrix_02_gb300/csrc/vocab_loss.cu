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
                           float* __restrict__ log_q) {
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

// Numbers the tokens that are learnt from, in order (one block).  Cross
// entropy also writes its one entry per token here.  Forward: loss and lse
// of the other tokens are 0.  Gradients: the power of two that brings the
// largest |g·τ| near 2^14 (binary16 G; 1 for bfloat16, whose exponents
// need no help).
__global__ void __launch_bounds__(1024)
    number_tokens_kernel(int T, int V, int top,
                         const int64_t* __restrict__ targets,
                         int* __restrict__ ids, float* __restrict__ log_q,
                         float* __restrict__ loss, float* __restrict__ lse,
                         const float* __restrict__ grad_loss,
                         long long grad_stride, float tau, int scaled,
                         int* __restrict__ token, int* __restrict__ row,
                         VocabHeader* header) {
  __shared__ int s_count[32];
  __shared__ float s_max[32];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int base = 0;
  float most = 0.f;
  for (int t0 = 0; t0 < T; t0 += 1024) {
    const int t = t0 + threadIdx.x;
    bool learnt = false;
    if (t < T) {
      if (targets) {
        const int64_t y = targets[t];
        learnt = y >= 0 && y < V;
        ids[t] = learnt ? (int)y : INT_MAX;
        log_q[t] = learnt ? 0.f : -INFINITY;
      } else {
        learnt = ids[(long long)t * top] != INT_MAX;
      }
    }
    const unsigned votes = __ballot_sync(0xffffffffu, learnt);
    if (lane == 0) s_count[warp] = __popc(votes);
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < 32; ++w) {
      const int c = s_count[w];
      if (w < warp) before += c;
      total += c;
    }
    const int r = base + before + __popc(votes & ((1u << lane) - 1u));
    if (t < T) {
      row[t] = learnt ? r : -1;
      if (learnt) token[r] = t;
      if (loss && !learnt) {
        loss[t] = 0.f;
        lse[t] = 0.f;
      }
      if (grad_loss && learnt)
        most = fmaxf(most, fabsf(grad_loss[t * grad_stride]));
    }
    base += total;
    __syncthreads();
  }
  for (int o = 16; o; o >>= 1)
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (lane == 0) s_max[warp] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 32; ++w) most = fmaxf(most, s_max[w]);
    most *= tau;
    int e = 0;
    // 0, Inf and NaN: no scale
    if (scaled && most > 0.f && most < INFINITY)
      e = min(max(14 - ilogbf(most), -100), 100);
    header->learnt = base;
    header->scale = ldexpf(1.f, e);
    header->inv_scale = ldexpf(1.f, -e);
  }
}

// ------------------------------------------------------------- products
// C (rows × cols) = A·B, one 64 × 64 tile per block, 4 × 4 per thread.
// Element (m, k) of A is A[rowA(m)·am + colA(k)·ak], where the map (token
// numbers) applies to whichever index walks X's rows; likewise B.
template <typename TA, typename TB>
struct Operand2 {
  const TA* A;
  long long am, ak;
  const int* map_m;  // A's row m is map_m[m]
  const TB* B;
  long long bk, bn;
  const int* map_k;  // B's row k is map_k[k]
};

// rows or depth < 0: the header's count of learnt tokens.
// out32 (+ add): fp32, C[m·ldc + n] (+)= sum.  out16: C = sum·inv_scale.
template <typename TA, typename TB, typename TO>
__global__ void __launch_bounds__(256)
    simple_product_kernel(Operand2<TA, TB> o, int rows, int cols, int depth,
                          const VocabHeader* header, TO* C, long long ldc,
                          int add) {
  __shared__ float sa[16][65], sb[16][65];
  griddep_wait();
  griddep_launch_dependents();
  if (rows < 0) rows = header->learnt;
  if (depth < 0) depth = header->learnt;
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  if (m0 >= rows) return;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < depth; k0 += 16) {
    for (int i = threadIdx.x; i < 1024; i += 256) {
      {
        const int k = o.ak == 1 ? i & 15 : i >> 6;
        const int m = o.ak == 1 ? i >> 4 : i & 63;
        float v = 0.f;
        if (m0 + m < rows && k0 + k < depth) {
          const long long mm = o.map_m ? o.map_m[m0 + m] : m0 + m;
          v = load_f(o.A + mm * o.am + (long long)(k0 + k) * o.ak);
        }
        sa[k][m] = v;
      }
      {
        const int k = o.bk == 1 ? i & 15 : i >> 6;
        const int n = o.bk == 1 ? i >> 4 : i & 63;
        float v = 0.f;
        if (n0 + n < cols && k0 + k < depth) {
          const long long kk = o.map_k ? o.map_k[k0 + k] : k0 + k;
          v = load_f(o.B + kk * o.bk + (long long)(n0 + n) * o.bn);
        }
        sb[k][n] = v;
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = sa[k][ty + 16 * i];
        b[i] = sb[k][tx + 16 * i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m < rows && n < cols) {
        TO* c = C + m * ldc + n;
        if constexpr (sizeof(TO) == 4)
          *c = add ? *c + acc[i][j] : acc[i][j];
        else
          store16(c, acc[i][j] * header->inv_scale);
      }
    }
}

// Softmax statistics of one piece of logits (columns v0 .. v0 + n), one
// block per row: running maximum and sum of exponentials, and the targets'
// logits (both over z/τ).
__global__ void __launch_bounds__(256)
    piece_stats_kernel(VocabTargets tg, const float* __restrict__ Z,
                       long long ldz, int v0, int n, float2* stats,
                       float* picked) {
  __shared__ float s_red[8];
  griddep_wait();
  griddep_launch_dependents();
  const int r = blockIdx.x;
  if (r >= tg.header->learnt) return;
  const int t = tg.token[r], warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float* z = Z + (long long)r * ldz;
  float m = -INFINITY;
  for (int i = threadIdx.x; i < n; i += 256) m = fmaxf(m, z[i] * tg.inv_tau);
  for (int o = 16; o; o >>= 1)
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) s_red[warp] = m;
  __syncthreads();
  for (int w = 0; w < 8; ++w) m = fmaxf(m, s_red[w]);
  const float2 old = v0 ? stats[r] : make_float2(-INFINITY, 0.f);
  const float peak = fmaxf(m, old.x);
  float s = 0.f;
  for (int i = threadIdx.x; i < n; i += 256)
    s += expf(z[i] * tg.inv_tau - peak);
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  __syncthreads();
  if (lane == 0) s_red[warp] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = old.y * expf(old.x - peak);
    for (int w = 0; w < 8; ++w) s += s_red[w];
    stats[r] = make_float2(peak, s);
  }
  for (int j = threadIdx.x; j < tg.top; j += 256) {
    const int id = tg.ids[(long long)t * tg.top + j];
    if (id >= v0 && id < v0 + n)
      picked[(long long)r * tg.top + j] = z[id - v0] * tg.inv_tau;
  }
}

// loss and lse of the learnt tokens, one thread each.
__global__ void __launch_bounds__(128)
    finish_loss_kernel(VocabTargets tg, const float2* __restrict__ stats,
                       const float* __restrict__ picked, float tau,
                       float* __restrict__ loss, float* __restrict__ lse) {
  griddep_wait();
  griddep_launch_dependents();
  const int r = blockIdx.x * blockDim.x + threadIdx.x;
  if (r >= tg.header->learnt) return;
  const int t = tg.token[r];
  const float2 st = stats[r];
  const float l = st.x + logf(st.y);
  float sum = 0.f;
  for (int j = 0; j < tg.top; ++j) {
    if (tg.ids[(long long)t * tg.top + j] == INT_MAX) break;
    const float lq = tg.log_q[(long long)t * tg.top + j];
    sum += expf(lq) * (lq - (picked[(long long)r * tg.top + j] - l));
  }
  loss[t] = tau * tau * sum;
  lse[t] = l;
}

// Z of one piece becomes G·scale in place, one block per row.
__global__ void __launch_bounds__(256)
    piece_grad_kernel(VocabTargets tg, float* __restrict__ Z, long long ldz,
                      int v0, int n, const float* __restrict__ lse,
                      const float* __restrict__ grad_loss,
                      long long grad_stride, float tau) {
  griddep_wait();
  griddep_launch_dependents();
  const int r = blockIdx.x;
  if (r >= tg.header->learnt) return;
  const int t = tg.token[r];
  float* z = Z + (long long)r * ldz;
  const float l = lse[t];
  const float g = grad_loss[t * grad_stride] * tau * tg.header->scale;
  for (int i = threadIdx.x; i < n; i += 256) {
    float p = expf(z[i] * tg.inv_tau - l);
    for (int j = 0; j < tg.top; ++j) {
      const int id = tg.ids[(long long)t * tg.top + j];
      if (id > v0 + i) break;
      if (id == v0 + i) p -= expf(tg.log_q[(long long)t * tg.top + j]);
    }
    z[i] = g * p;
  }
}

// dX row by row: the sum over the pieces, rounded; zeros for the tokens
// that are not learnt from.
template <typename T16>
__global__ void __launch_bounds__(256)
    finish_dx_kernel(int T, int D, const int* __restrict__ row,
                     const VocabHeader* header,
                     const float* __restrict__ sum, T16* __restrict__ dX,
                     long long lddx) {
  griddep_wait();
  griddep_launch_dependents();
  const int t = blockIdx.x;
  const int r = row[t];
  for (int i = threadIdx.x; i < D; i += 256)
    store16(dX + t * lddx + i,
            r < 0 ? 0.f : sum[(long long)r * D + i] * header->inv_scale);
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

// Where a call's state lies in its workspace.
struct VocabLayout {
  int64_t piece;  // columns of a piece
  int64_t header, token, row, ids, log_q, stats, picked, z, dx, total;
};

VocabLayout layout(int64_t T, int64_t V, int64_t D, int64_t top, bool grad) {
  VocabLayout l = {};
  const int64_t most = 64ll << 20;  // logits of a piece
  l.piece = std::min(up(V, 64),
                     std::max<int64_t>(64, most / std::max<int64_t>(T, 1) /
                                               64 * 64));
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += up(bytes, 256);
    return here;
  };
  l.header = take(sizeof(VocabHeader));
  l.token = take(T * 4);
  l.row = take(T * 4);
  l.ids = take(T * top * 4);
  l.log_q = take(T * top * 4);
  l.z = take(T * l.piece * 4);
  if (grad) {
    l.dx = take(T * D * 4);
  } else {
    l.stats = take(T * 8);
    l.picked = take(T * top * 4);
  }
  l.total = at;
  return l;
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

template <typename T16>
cudaError_t run_typed(const VocabCall& c, bool grad, const WaitCfg&) {
  const int T = (int)c.T, V = (int)c.V, D = (int)c.D, top = (int)c.top;
  cudaStream_t s = c.stream;
  const VocabLayout l = layout(c.T, c.V, c.D, c.top, grad);
  char* ws = static_cast<char*>(c.ws);
  auto* header = reinterpret_cast<VocabHeader*>(ws + l.header);
  int* token = reinterpret_cast<int*>(ws + l.token);
  int* row = reinterpret_cast<int*>(ws + l.row);
  int* ids = reinterpret_cast<int*>(ws + l.ids);
  float* log_q = reinterpret_cast<float*>(ws + l.log_q);
  float* z = reinterpret_cast<float*>(ws + l.z);
  const T16* X = static_cast<const T16*>(c.X);
  const T16* W = static_cast<const T16*>(c.W);
  cudaError_t e;
  const float inv_tau = 1.f / c.tau;
  if (!c.targets && T > 0) {
    e = launch_pdl(distill_targets_kernel,
                   dim3((T + kTargetWarps - 1) / kTargetWarps),
                   dim3(32 * kTargetWarps), 0, s, T, V, top, c.top_logits,
                   (long long)c.ldt, c.top_ids, (long long)c.ldi, inv_tau,
                   ids, log_q);
    if (e != cudaSuccess) return e;
  }
  e = launch_pdl(number_tokens_kernel, dim3(1), dim3(1024), 0, s, T, V, top,
                 c.targets, ids, log_q, c.loss, c.lse, c.grad_loss,
                 (long long)c.grad_stride, c.tau,
                 c.type == GEMM_F32_MIXED_F16 ? 1 : 0, token, row, header);
  if (e != cudaSuccess) return e;
  const VocabTargets tg{header, token, row, ids, log_q, top, inv_tau};
  float* sum = reinterpret_cast<float*>(ws + l.dx);
  float2* stats = reinterpret_cast<float2*>(ws + l.stats);
  float* picked = reinterpret_cast<float*>(ws + l.picked);
  const unsigned rows64 = (T + 63) / 64, cols64 = (D + 63) / 64;
  for (int64_t v0 = 0; v0 < c.V; v0 += l.piece) {
    const int n = (int)std::min(l.piece, c.V - v0);
    const T16* Wp = W + v0 * c.ldw;
    if (T > 0) {
      const Operand2<T16, T16> logits{X, c.ldx, 1, token,
                                      Wp, 1, c.ldw, nullptr};
      e = launch_pdl(simple_product_kernel<T16, T16, float>,
                     dim3((n + 63) / 64, rows64), dim3(256), 0, s, logits, -1,
                     n, D, header, z, (long long)l.piece, 0);
      if (e != cudaSuccess) return e;
    }
    if (!grad) {
      e = launch_pdl(piece_stats_kernel, dim3(T), dim3(256), 0, s, tg, z,
                     (long long)l.piece, (int)v0, n, stats, picked);
      if (e != cudaSuccess) return e;
      continue;
    }
    if (T > 0) {
      e = launch_pdl(piece_grad_kernel, dim3(T), dim3(256), 0, s, tg, z,
                     (long long)l.piece, (int)v0, n, c.lse_in, c.grad_loss,
                     (long long)c.grad_stride, c.tau);
      if (e != cudaSuccess) return e;
      const Operand2<float, T16> back{z, l.piece, 1, nullptr,
                                      Wp, c.ldw, 1, nullptr};
      e = launch_pdl(simple_product_kernel<float, T16, float>,
                     dim3(cols64, rows64), dim3(256), 0, s, back, -1, D, n,
                     header, sum, (long long)D, v0 ? 1 : 0);
      if (e != cudaSuccess) return e;
    }
    const Operand2<float, T16> outer{z, 1, l.piece, nullptr,
                                     X, c.ldx, 1, token};
    e = launch_pdl(simple_product_kernel<float, T16, T16>,
                   dim3(cols64, (n + 63) / 64), dim3(256), 0, s, outer, n, D,
                   -1, header, static_cast<T16*>(c.dW) + v0 * c.lddw,
                   (long long)c.lddw, 0);
    if (e != cudaSuccess) return e;
  }
  if (T == 0) return cudaSuccess;
  if (!grad)
    return launch_pdl(finish_loss_kernel, dim3((T + 127) / 128), dim3(128), 0,
                      s, tg, stats, picked, c.tau, c.loss, c.lse);
  return launch_pdl(finish_dx_kernel<T16>, dim3(T), dim3(256), 0, s, T, D,
                    row, header, sum, static_cast<T16*>(c.dX),
                    (long long)c.lddx);
}

int run_vocab(const VocabCall& c, bool grad, bool distill) {
  int st = check_call(c, grad, distill);
  if (st != GEMM_F32_OK) return st;
  if (c.T == 0 && !grad) return GEMM_F32_OK;
  const VocabLayout l = layout(c.T, c.V, c.D, c.top, grad);
  if (!c.ws || (reinterpret_cast<uintptr_t>(c.ws) & 15u) != 0 ||
      c.ws_bytes < l.total)
    return GEMM_F32_ERR_INVALID_ARG;
  int sms = 0, cc = 0;
  WaitCfg wc;
  cudaError_t e = device_facts(&sms, &cc, &wc);
  if (e != cudaSuccess) return record_cuda_error(e);
  if (cc != 10) return GEMM_F32_ERR_UNSUPPORTED;
  e = c.type == GEMM_F32_MIXED_BF16 ? run_typed<__nv_bfloat16>(c, grad, wc)
                                    : run_typed<__half>(c, grad, wc);
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
  return layout(T, V, D, top, grad != 0).total;
}

}  // extern "C"
