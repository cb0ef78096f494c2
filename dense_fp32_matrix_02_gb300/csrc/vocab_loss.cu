// Vocabulary losses: softmax cross entropy and distillation of z = X·Wᵀ,
// forward and backward (the definitions are in include/gemm_f32.h).
//
// Both losses are one computation.  Token t has a sparse target distribution
// q_t (one entry for cross entropy, the teacher's softmax over its entries
// for distillation) and, with p_t = softmax(z_t/τ),
//   loss_t = τ²·Σ_j q_tj·(log q_tj − (z[t][id_tj]/τ − lse_t)),
//   dL/dz_t = g_t·τ·(p_t − q_t)
// (cross entropy: q = 1, τ = 1).  A call runs
//   1. the targets: entries sorted by id with log q or q; the tokens that are
//      learnt from, numbered (everything after works on those rows only);
//   2. forward: the logits piece by piece, each reduced to per-row softmax
//      statistics and the targets' logits; then loss and lse;
//      backward: each piece made again, turned into G = dL/dz, and
//      multiplied by W (dX, added up over the pieces) and by X (dW's rows
//      of that piece).
#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <type_traits>

#include "gemm_f32.h"
#include "kernels.h"
#include "vocab.cuh"

namespace gemm_f32_impl {
namespace {

// ------------------------------------------------------------- targets
// Distillation: one warp per token.  log q (forward) or q over the entries
// that count, which are ranked by (id, place) and written in that order.
constexpr int kTargetWarps = 4;

__global__ void __launch_bounds__(32 * kTargetWarps)
    distill_targets_kernel(int T, int V, int top,
                           const float* __restrict__ logits, long long ldt,
                           const int64_t* __restrict__ top_ids, long long ldi,
                           float inv_tau, int logs, int* __restrict__ ids,
                           float* __restrict__ weights,
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
      const float log_q = (u[i] - peak) - log_sum;
      weights[(long long)t * top + rank] = logs ? log_q : expf(log_q);
    }
  }
}

// Numbers the tokens that are learnt from, in order, and packs their rows of
// X where they are not read in place (some token is not learnt from, or X
// has no tensor map); packs W's rows where they have no tensor map.  Every block numbers all tokens, 256 a warp at a time
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
  int D;
  int share;        // tokens of a block
  const uint16_t* W;  // where it has no tensor map, else null
  long long ldw;
  uint16_t* Wp;
  // gradients
  int piece, pieces, pairs;
  long long slot_rows;  // of dX's slots, all together
  int dw_max_splits;
  int* tile_slots;      // slots of each tile of dX
};

// The shares of dX's steps (VocabShare), a pair a thread: each pair's is what
// its tiles of G and dW leave of an even total, in stretches that keep a
// tile's slots within the room for them and no share under eight steps.  The
// first `more_w` pairs have one tile of dW more than the others, the last
// `more_g` one of G; so the pairs fall into three runs with one room each,
// and everything has a closed form.  (All step counts are below 2^30: the
// host checks.)
struct Shares {
  int line, left, cut;  // steps of a tile; of the line; of a stretch
  int end0, end1;       // ends of the first and second run of pairs
  int room0, room1, room2;
  __device__ __forceinline__ int end(int p, int pairs) const {
    // (to the pair's end, inclusive)
    const int q = p + 1;
    long long sum = (long long)min(q, end0) * room0 +
                    (long long)max(0, min(q, end1) - end0) * room1 +
                    (long long)max(0, q - end1) * room2;
    if (sum >= left || q == pairs) return left;
    const int x = (int)sum, tile = x / line, k = x - tile * line;
    return tile * line + min(line, (k + cut / 2) / cut * cut);
  }
};

__device__ void share_out(const NumberArgs& a, int learnt, int dw_splits,
                          VocabHeader* header) {
  const int p = threadIdx.x, pairs = a.pairs;
  if (p >= pairs) return;
  const int tiles = vocab_tiles(learnt) * vocab_tiles(a.D);
  const int tall = vocab_tiles(a.piece), line = vocab_steps(a.piece);
  const int tiles_w = tall * vocab_tiles(a.D) * dw_splits;
  const int tiles_g = a.pieces > 1 ? vocab_tiles(learnt) * tall : 0;
  const int cost_w = vocab_tile_cost(vocab_steps(learnt) / dw_splits);
  const int cost_g = vocab_tile_cost(vocab_steps(a.D));
  const int more_w = tiles_w % pairs, more_g = tiles_g % pairs;
  const int base = tiles_w / pairs * cost_w + tiles_g / pairs * cost_g;
  Shares s;
  s.end0 = min(more_w, pairs - more_g);
  s.end1 = max(more_w, pairs - more_g);
  const bool both = more_w > pairs - more_g;
  const int c0 = more_w ? cost_w : 0, c2 = more_g ? cost_g : 0;
  const int c1 = both ? cost_w + cost_g : 0;
  const int n0 = s.end0, n1 = s.end1 - s.end0, n2 = pairs - s.end1;
  // the level over `base` at which the room under it holds all steps
  const long long all = (long long)tiles * line;
  int level = INT_MAX;
#pragma unroll 1
  for (int round = 0; round < 4; ++round) {
    long long sum = all;
    int count = 0;
    if (n0 && c0 < level) sum += (long long)n0 * c0, count += n0;
    if (n1 && c1 < level) sum += (long long)n1 * c1, count += n1;
    if (n2 && c2 < level) sum += (long long)n2 * c2, count += n2;
    const int now = (int)(((double)sum + count - 1) / count);
    if (now >= level) break;
    level = now;
  }
  s.room0 = max(0, level - c0);
  s.room1 = max(0, level - c1);
  s.room2 = max(0, level - c2);
  // whole rounds: what the fullest pair has room for
  int least = INT_MAX;
  if (n0) least = s.room0;
  if (n1) least = min(least, s.room1);
  if (n2) least = min(least, s.room2);
  const int rounds = min(least / line, tiles / pairs), whole = rounds * pairs;
  s.room0 -= rounds * line;
  s.room1 -= rounds * line;
  s.room2 -= rounds * line;
  s.line = line;
  s.left = (tiles - whole) * line;
  const int most = (int)max(
      1ll, min(1ll << 30, a.slot_rows / vocab_slot_rows(learnt)));
  s.cut = max((line + most - 1) / most, min(line, 8));
  if (p == 0) header->dx_rounds = rounds;
  for (int tile = p; tile < whole; tile += pairs) a.tile_slots[tile] = 1;
  VocabShare sh;
  sh.x0 = p ? s.end(p - 1, pairs) : 0;
  sh.x1 = s.end(p, pairs);
  sh.slot = 0;
  if (sh.x1 > sh.x0) {
    const int first = sh.x0 / line, start = first * line;
    int next = sh.x0;  // the ends before this pair's, backwards
#pragma unroll 1
    for (int j = p - 1; j >= 0 && next > start; --j) {
      const int begin = j ? s.end(j - 1, pairs) : 0;
      sh.slot += next > begin;
      next = begin;
    }
    // the tiles that end with this share
    int slot = sh.slot;
    for (int tile = first; (tile + 1) * line <= sh.x1; ++tile, slot = 0)
      a.tile_slots[whole + tile] = slot + 1;
  }
  header->share[p] = sh;
}

// 16-bit row of n elements, then zeros up to a multiple of 8, to a 16-byte
// aligned row; by one warp.  vec: the source is 16-byte aligned too; else it
// is read in the aligned 4-byte words that hold it (a word that lies partly
// outside the row is read as single elements).
__device__ __forceinline__ void pack_row(const uint16_t* __restrict__ src,
                                         int n, uint16_t* __restrict__ dst,
                                         bool vec, int lane) {
  const int odd = (reinterpret_cast<uintptr_t>(src) >> 1) & 1;
  for (int c = 8 * lane; c < n; c += 256) {
    uint4 v;
    if (vec && c + 8 <= n) {
      v = *reinterpret_cast<const uint4*>(src + c);
    } else if (c >= odd && c + 8 + odd <= n) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(src + c - odd);
      const uint32_t a = w[0], b = w[1], d = w[2], e = w[3];
      v = make_uint4(a, b, d, e);
      if (odd) {
        v.x = __funnelshift_r(a, b, 16);
        v.y = __funnelshift_r(b, d, 16);
        v.z = __funnelshift_r(d, e, 16);
        v.w = __funnelshift_r(e, w[4], 16);
      }
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
                         float* __restrict__ weights, int* __restrict__ token,
                         int* __restrict__ row, VocabHeader* header) {
  __shared__ int s_count[32];
  __shared__ float s_max[32];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (a.W) {
    const int warps = gridDim.x * 32;
    for (long long v = blockIdx.x * 32 + warp; v < a.V; v += warps)
      pack_row(a.W + v * a.ldw, a.D, a.Wp + v * a.ldxp, false, lane);
  }
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
          weights[t] = a.loss ? 0.f : 1.f;  // log q, or q
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
    header->scale = ldexpf(1.f, e);
    header->inv_scale = ldexpf(1.f, -e);
  }
  if (!a.grad_loss) return;
  const int splits =
      vocab_dw_splits(base, a.piece, a.D, a.pairs, a.dw_max_splits);
  if (threadIdx.x == 0) header->dw_splits = splits;
  if (base > 0) {
    share_out(a, base, splits, header);
  } else if (threadIdx.x < a.pairs) {
    header->share[threadIdx.x] = VocabShare{0, 0, 0};
    header->dx_rounds = 0;
  }
}

// ------------------------------------------------------------- results
__device__ __forceinline__ float2 merge_stats(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  const float ref = m == -INFINITY ? 0.f : m;
  return make_float2(m, a.y * exp2f(a.x - ref) + b.y * exp2f(b.x - ref));
}

// loss and lse of the learnt tokens: 8 rows a block, blockDim / 8 threads a
// row that share out its statistics (parts of them, [part][T]) and join them
// in a fixed order.
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
      lq = tg.weights[t * tg.top + (lane >> 3)];
      at = picked[(long long)r * tg.top + (lane >> 3)];
    }
  }
  float2 st = make_float2(-INFINITY, 0.f);
  if (here) {
#pragma unroll 4
    for (int e = slice; e < parts; e += blockDim.x >> 3)
      st = merge_stats(st, stats[(long long)e * T + r]);
  }
  for (int o = 8; o < 32; o <<= 1)
    st = merge_stats(st, make_float2(__shfl_xor_sync(0xffffffffu, st.x, o),
                                     __shfl_xor_sync(0xffffffffu, st.y, o)));
  const int warps = blockDim.x >> 5;
  if (warps > 1) {
    if (lane < 8) s_part[warp][lane] = st;
    __syncthreads();
    if (warp > 0) return;
    st = make_float2(-INFINITY, 0.f);
    for (int w = lane >> 3; w < warps; w += 4)
      st = merge_stats(st, s_part[w][lane & 7]);
    for (int o = 8; o < 32; o <<= 1)
      st = merge_stats(st, make_float2(__shfl_xor_sync(0xffffffffu, st.x, o),
                                       __shfl_xor_sync(0xffffffffu, st.y, o)));
  }
  const float l = st.x * 0.69314718f + logf(st.y);
  float sum = 0.f;
  for (int j = lane >> 3; id != INT_MAX;) {
    sum += expf(lq) * (lq - (at - l));
    j += 4;
    if (j >= tg.top) break;
    id = tg.ids[t * tg.top + j];
    lq = tg.weights[t * tg.top + j];
    at = picked[(long long)r * tg.top + j];
  }
  for (int o = 8; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (here && lane < 8) {
    loss[t] = tau * tau * sum;
    lse[t] = l;
  }
}

// dX, four columns a thread: the sum of its tiles' slots in order, rounded;
// zeros for the tokens that are not learnt from.  vec: dX's rows are 8-byte
// aligned.
template <typename T16>
__global__ void __launch_bounds__(256)
    finish_dx_kernel(int T, int D, const int* __restrict__ row,
                     const VocabHeader* __restrict__ header,
                     const int* __restrict__ tile_slots,
                     const float* __restrict__ slots, long long ld_slot,
                     T16* __restrict__ dX, long long lddx, int vec) {
  griddep_wait();
  griddep_launch_dependents();
  const int learnt = header->learnt;
  const float inv_scale = header->inv_scale;
  const long long next = vocab_slot_rows(learnt) * ld_slot;
  const int chunks = (int)(ld_slot / 4), wide = vocab_tiles(D);
  const long long total = (long long)T * chunks;
  for (long long k = blockIdx.x * 256ll + threadIdx.x; k < total;
       k += gridDim.x * 256ll) {
    const long long t = k / chunks;
    const int i = (int)(k - t * chunks) * 4;
    const int r = learnt == T ? (int)t : row[t];
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r >= 0) {
      // this tile's place in the order of the line (tile_coords)
      const int tm = r / kVocabTile, group = tm / kVocabGroup * kVocabGroup;
      const int high = min(vocab_tiles(learnt) - group, kVocabGroup);
      const int n =
          tile_slots[group * wide + i / kVocabTile * high + (tm - group)];
      const float* from = slots + (long long)r * ld_slot + i;
      for (int s0 = 0; s0 < n; s0 += 8) {
        float4 a[8];
#pragma unroll
        for (int s = 0; s < 8; ++s)
          a[s] = s0 + s < n ? *reinterpret_cast<const float4*>(
                                  from + (s0 + s) * next)
                            : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          v.x += a[s].x;
          v.y += a[s].y;
          v.z += a[s].z;
          v.w += a[s].w;
        }
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

// A piece's rows of dW where they were summed in slots, rounded.
template <typename T16>
__global__ void __launch_bounds__(256)
    finish_dw_kernel(int n, int D, const VocabHeader* __restrict__ header,
                     const float* __restrict__ slots, long long slot_rows,
                     long long ld_slot, T16* __restrict__ dW, long long lddw) {
  griddep_wait();
  griddep_launch_dependents();
  const int splits = header->dw_splits;
  if (splits == 1) return;
  const float inv_scale = header->inv_scale;
  const int chunks = (int)(ld_slot / 4);
  for (long long k = blockIdx.x * 256ll + threadIdx.x;
       k < (long long)n * chunks; k += gridDim.x * 256ll) {
    const long long r = k / chunks;
    const int i = (int)(k - r * chunks) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      const float4 a = *reinterpret_cast<const float4*>(
          slots + (s * slot_rows + r) * ld_slot + i);
      v.x += a.x;
      v.y += a.y;
      v.z += a.z;
      v.w += a.w;
    }
    T16* to = dW + r * lddw + i;
    const float o[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < D) store16(to + j, o[j] * inv_scale);
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
  int64_t piece, pieces;  // columns of G
  int64_t ld_pack;        // row stride of the packed copies
  int64_t ld_slot;        // row stride of the fp32 slots
  int64_t slot_rows;      // dX's slots, all together
  int64_t dw_slot_rows, dw_max_splits;  // dW's; 1: none
  int64_t header, token, row, flags, ids, weights, x_pack, w_pack, total;
  int64_t stats, picked;                    // forward
  int64_t g[2], tile_slots, slots, dw_slots;  // gradients
};

VocabLayout layout(int64_t T, int64_t V, int64_t D, int64_t top, bool grad,
                   bool pack_w) {
  int64_t kMostG = 128ll << 20;
  if (const char* env = std::getenv("VOCAB_PIECE_MB"))
    kMostG = (int64_t)std::atoi(env) << 20;
  constexpr int64_t kMostSlots = 768ll << 20;
  constexpr int64_t kMostDwSlots = 128ll << 20;
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
  l.weights = take(rows * top * 4);
  l.x_pack = take(up(rows, 64) * l.ld_pack * 2);
  if (pack_w) l.w_pack = take(V * l.ld_pack * 2);
  if (grad) {
    // equal pieces, whole tiles, of at most kMostG bytes of G
    const int64_t widest = std::max<int64_t>(
        kVocabTile, kMostG / (2 * rows) / kVocabTile * kVocabTile);
    l.pieces = (V + widest - 1) / widest;
    l.piece = up((V + l.pieces - 1) / l.pieces, kVocabTile);
    l.pieces = (V + l.piece - 1) / l.piece;
    l.ld_slot = up(D, 4);
    const int64_t slot = up(rows, kVocabTile) * l.ld_slot * 4;
    l.slot_rows = up(rows, kVocabTile) *
                  std::min<int64_t>(kVocabMaxPairs,
                                    std::max<int64_t>(1, kMostSlots / slot));
    l.g[0] = take(rows * l.piece * 2);
    l.g[1] = l.pieces > 1 ? take(rows * l.piece * 2) : l.g[0];
    l.tile_slots = take((int64_t)vocab_tiles(rows) * vocab_tiles(D) * 4);
    l.slots = take(l.slot_rows * l.ld_slot * 4);
    l.dw_slot_rows = up(std::min(l.piece, V), 32);
    l.dw_max_splits = 1;
    if ((int64_t)vocab_tiles(l.piece) * vocab_tiles(D) < kVocabMaxPairs)
      l.dw_max_splits = std::min<int64_t>(
          kVocabMaxDwSplits,
          std::max<int64_t>(
              1, kMostDwSlots / (l.dw_slot_rows * l.ld_slot * 4)));
    if (l.dw_max_splits > 1)
      l.dw_slots = take(l.dw_max_splits * l.dw_slot_rows * l.ld_slot * 4);
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
  float* weights = reinterpret_cast<float*>(ws + l.weights);
  const float inv_tau = 1.f / c.tau;
  cudaError_t e;

  auto* flags = reinterpret_cast<uint8_t*>(ws + l.flags);
  if (!c.targets) {
    e = launch_pdl(distill_targets_kernel,
                   dim3((T + kTargetWarps - 1) / kTargetWarps),
                   dim3(32 * kTargetWarps), 0, s, T, V, top, c.top_logits,
                   (long long)c.ldt, c.top_ids, (long long)c.ldi, inv_tau,
                   grad ? 0 : 1, ids, weights, flags);
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
  na.D = D;
  na.piece = (int)std::min(l.piece, c.V), na.pieces = (int)l.pieces;
  na.pairs = vocab_pairs(sms), na.slot_rows = l.slot_rows;
  na.dw_max_splits = (int)l.dw_max_splits;
  na.tile_slots = reinterpret_cast<int*>(ws + l.tile_slots);
  if (!w_fits) {
    na.W = static_cast<const uint16_t*>(c.W), na.ldw = c.ldw;
    na.Wp = reinterpret_cast<uint16_t*>(ws + l.w_pack);
  }
  const int blocks = w_fits ? std::min(sms, (T + 31) / 32) : sms;
  na.share = (T + blocks - 1) / blocks;
  e = launch_pdl(number_tokens_kernel, dim3(blocks), dim3(1024), 0, s, na, ids,
                 weights, token, row, header);
  if (e != cudaSuccess) return e;
  const char* W = w_fits ? static_cast<const char*>(c.W) : ws + l.w_pack;
  const int64_t ldw = w_fits ? c.ldw : l.ld_pack;

  VocabGemm p = {};
  p.type = c.type;
  p.T = T, p.D = D;
  p.X = c.X, p.ldx = c.ldx;
  p.Xp = ws + l.x_pack, p.ldxp = l.ld_pack, p.rows_xp = (int)up(c.T, 64);
  p.W = W, p.ldw = ldw;
  p.V = V;
  p.targets = VocabTargets{header, token, ids, weights, top, inv_tau};
  if (!grad) {
    p.stats = reinterpret_cast<float2*>(ws + l.stats);
    p.picked = reinterpret_cast<float*>(ws + l.picked);
    if ((e = launch_vocab_stats(p, sms, wc, s)) != cudaSuccess) return e;
    // a thread's share of a row: about four statistics, in one warp's reach
    // of 128 threads
    const int parts = (V + 127) / 128;
    const int threads = parts <= 16 ? 32 : parts <= 128 ? 256 : 1024;
    return launch_pdl(finish_loss_kernel, dim3((T + 7) / 8), dim3(threads), 0,
                      s, p.targets, T, parts, p.stats, p.picked, c.tau, c.loss,
                      c.lse);
  }
  p.piece = na.piece, p.ldg = l.piece;
  p.lse = c.lse_in;
  p.grad_loss = c.grad_loss, p.grad_stride = c.grad_stride, p.tau = c.tau;
  p.slots = reinterpret_cast<float*>(ws + l.slots);
  p.slot_rows = l.slot_rows, p.ld_slot = l.ld_slot;
  if (l.dw_max_splits > 1)
    p.dw_slots = reinterpret_cast<float*>(ws + l.dw_slots);
  p.dw_slot_rows = l.dw_slot_rows, p.dw_max_splits = (int)l.dw_max_splits;
  p.dW = c.dW, p.lddw = c.lddw;
  auto piece_at = [&](int64_t i) {
    if (i < 0 || i >= l.pieces) return VocabPiece{0, 0, nullptr};
    const int64_t v0 = i * l.piece;
    return VocabPiece{(int)v0, (int)std::min(l.piece, c.V - v0),
                      ws + l.g[i & 1]};
  };
  auto finish = [&](auto* dX) -> cudaError_t {
    using T16 = std::remove_pointer_t<decltype(dX)>;
    for (int64_t i = 0; i <= l.pieces; ++i) {
      p.grad = piece_at(i), p.back = piece_at(i - 1);
      p.first = i == 1;
      if ((e = launch_vocab_step(p, sms, wc, s)) != cudaSuccess) return e;
      if (i > 0 && p.dw_slots) {
        e = launch_pdl(finish_dw_kernel<T16>, dim3(2 * sms), dim3(256), 0, s,
                       p.back.n, D, header, p.dw_slots, p.dw_slot_rows,
                       p.ld_slot,
                       static_cast<T16*>(c.dW) + p.back.v0 * c.lddw,
                       (long long)c.lddw);
        if (e != cudaSuccess) return e;
      }
    }
    const int vec = (reinterpret_cast<uintptr_t>(c.dX) & 7u) == 0 &&
                    c.lddx % 4 == 0;
    const int64_t groups = (c.T * (l.ld_slot / 4) + 255) / 256;
    return launch_pdl(finish_dx_kernel<T16>,
                      dim3((unsigned)std::min<int64_t>(groups, 8ll * sms)),
                      dim3(256), 0, s, T, D, row, header, na.tile_slots, p.slots, p.ld_slot, dX,
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
  // tiles, and all steps of a piece's products, are counted in 32 bits
  const int64_t wide = up(c.D, kVocabTile) / kVocabTile;
  const int64_t rows = up(c.T, kVocabTile) / kVocabTile;
  if ((rows + l.piece) * wide > (1 << 30) ||
      rows * wide * (l.piece / 64 + 1) > (1 << 30) ||
      rows * (c.V / kVocabTile + 1) > (1 << 30))
    return GEMM_F32_ERR_UNSUPPORTED;
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
