// Vocabulary losses and log probabilities: softmax cross entropy and
// distillation of z = X·Wᵀ, the log probabilities of given words with entropy
// and the likeliest others, forward and backward (the definitions are in
// include/gemm_f32.h): argument checks, workspace and launch.
//
// Both losses are one computation.  Token t has a sparse target distribution
// q_t (one entry for cross entropy, the teacher's softmax over its entries
// for distillation) and, with p_t = softmax(z_t/τ),
//   loss_t = τ²·Σ_j q_tj·(log q_tj − (z[t][id_tj]/τ − lse_t)),
//   dL/dz_t = g_t·τ·(p_t − q_t)
// (cross entropy: q = 1, τ = 1).  The forward call reduces each tile of the
// logits to softmax statistics and the targets' logits as it is made; the
// gradients make each piece of the logits again, turn it into G = dL/dz, and
// multiply it by W (dX, added up over the pieces) and by X (dW's rows of
// that piece).  A call runs
//   1. the targets: a teacher's entries sorted by id with log q or q; the
//      tokens that are learnt from, numbered (everything after works on
//      those rows only);
//   2. the products (vocab_gemm.cu);
//   3. the results from the products' partial ones.
// Log probabilities are cross entropy with more results, and with the logits
// kept for the gradients (vocab_score.cu).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "gemm_f32.h"
#include "kernels.h"
#include "vocab.cuh"

namespace gemm_f32_impl {
namespace {

// ------------------------------------------------------------- targets
// Distillation: a token to a group of lanes, the smallest power of two that
// gives each entry one (32 lanes for more).  log q (forward) or q over the
// entries that count, which are ranked by (id, place) and written in that
// order.  The largest logit is subtracted before the division by τ: a logit
// that stands for a mask, the type's lowest value, would overflow in it
// (τ < 1) and count as no entry here, but as one where ids are read.
constexpr int kTeacherWarps = 4;

__global__ void __launch_bounds__(32 * kTeacherWarps)
    teacher_kernel(const __grid_constant__ VocabCall p, int logs) {
  __shared__ int s_id[kTeacherWarps][kVocabMaxTop];
  griddep_wait();
  griddep_launch_dependents();
  constexpr int kPer = kVocabMaxTop / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* sid = s_id[warp];
  int wide = 1;
  while (wide < p.top && wide < 32) wide <<= 1;
  const int in = lane & (wide - 1), group = lane / wide, groups = 32 / wide;
  int* mine = sid + group * (kVocabMaxTop / groups);
  const long long t =
      ((long long)blockIdx.x * kTeacherWarps + warp) * groups + group;
  const bool here = t < p.T;
  float u[kPer];
  float peak = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int j = in + 32 * i;
    u[i] = -INFINITY;
    if (j < p.top && here) {
      const float l = p.top_logits[t * p.ldt + j];
      const int64_t id = p.top_ids[t * p.ldi + j];
      const bool counts = id >= 0 && id < p.V && l != -INFINITY;
      mine[j] = counts ? (int)id : INT_MAX;
      if (counts) u[i] = l;
      peak = fmaxf(peak, u[i]);
    }
  }
  for (int o = wide >> 1; o; o >>= 1)
    peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, o));
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (u[i] != -INFINITY) {  // (no entry)
      u[i] = (u[i] - peak) * p.inv_tau;
      sum += expf(u[i]);
    }
  for (int o = wide >> 1; o; o >>= 1)
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float log_sum = logf(sum);
  // sum is 0 only where nothing counts (the largest term is 1, or NaN)
  if (in == 0 && here) p.learnt_flag[t] = sum != 0.f;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int j = in + 32 * i;
    if (j < p.top && here) {
      const int id = mine[j];
      int rank = 0, prev = -1;  // prev: the id of the rank before
      for (int k = 0; k < p.top; ++k) {
        const int other = mine[k];
        if (other < id || (other == id && k < j)) {
          ++rank;
          prev = max(prev, other);
        }
      }
      const float log_q = u[i] - log_sum;
      if (!span_ok(p.ids + t * p.top + rank, 4, p.ids, 4ll * p.T * p.top,
                   p.status))
        continue;
      p.ids[t * p.top + rank] = id;
      p.weights[t * p.top + rank] = logs ? log_q : expf(log_q);
      // the blocks of 128 columns that start behind the entry before
      uint32_t* starts = p.starts + t * p.blocks;
      const int last = id == INT_MAX ? p.blocks - 1 : id >> 7;
      for (int b = (prev >> 7) + 1; b <= last; ++b)
        starts[b] = rank | (id != INT_MAX && b == last ? id & 127
                                                       : kVocabNone) << 16;
      if (rank == p.top - 1)
        for (int b = last + 1; b < p.blocks; ++b)
          starts[b] = p.top | kVocabNone << 16;
    }
  }
}

// Rows first, first + stride, ... below `rows` of src, or those of them that
// `to` numbers (to[row] >= 0: the row's place in dst), to 16-byte aligned
// rows; a warp each, four chunks of 16 bytes a lane at a time.
__device__ __forceinline__ void pack_rows(const uint16_t* src, long long lds,
                                          int n, uint16_t* dst, long long ldd,
                                          const int* to, bool vec,
                                          long long first, long long rows,
                                          int stride, int lane) {
  constexpr int kAhead = 4;
  const int chunks = (n + 7) / 8;
  long long r = first;
  int c = lane;
  while (r < rows) {
    uint4 v[kAhead];
    uint16_t* out[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      while (c >= chunks && r < rows) {
        r += stride;
        c = lane;  // (lanes past the last chunk sit a row out)
        if (c >= chunks) break;
      }
      out[a] = nullptr;
      if (r < rows && c < chunks) {
        const int at = to ? to[r] : 0;
        if (at >= 0) {
          out[a] = dst + (to ? at : r) * ldd + 8 * c;
          v[a] = read_8(src + r * lds, 8 * c, n, vec);
        }
      }
      c += 32;
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (out[a]) *reinterpret_cast<uint4*>(out[a]) = v[a];
  }
}

// The same for long rows that start off 16-byte boundaries: a warp reads a row
// in the aligned 16-byte pieces that hold it, and each lane puts its chunk
// together from its own piece and the next lane's.  (In 4-byte words, of which
// each lane reads five 16 bytes apart from the next lane's, rows of 2045
// elements went at 4.7 TB/s: 100000 of them 173 us.)  A piece that lies partly
// outside the row is read as single elements.
constexpr int kLongRow = 64;  // chunks
__device__ __forceinline__ void pack_long_rows(
    const uint16_t* src, long long lds, int n, uint16_t* dst, long long ldd,
    const int* to, long long first, long long rows, int stride, int lane) {
  constexpr int kAhead = 4;
  const int chunks = (n + 7) / 8;
  for (long long r = first; r < rows; r += stride) {
    const int at = to ? to[r] : 0;
    if (at < 0) continue;
    const uint16_t* row = src + r * lds;
    uint16_t* out = dst + (to ? at : r) * ldd;
    const int off = (reinterpret_cast<uintptr_t>(row) & 15u) >> 1;  // elements
    const bool two = off & 4, one = off & 2;
    const int bits = (off & 1) * 16;
    // piece j: elements 8·j - off and on
    auto piece = [&](int j) {
      const int e = 8 * j - off;
      if (e >= 0 && e + 8 <= n)
        return *reinterpret_cast<const uint4*>(row + e);
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i >= 0 && e + i < n)
          w[i >> 1] |= (uint32_t)row[e + i] << (16 * (i & 1));
      return make_uint4(w[0], w[1], w[2], w[3]);
    };
    for (int j0 = 0; j0 < chunks; j0 += 32 * kAhead) {
      uint4 v[kAhead], last[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int j = j0 + 32 * a + lane;
        v[a] = last[a] = make_uint4(0, 0, 0, 0);
        if (j < chunks) v[a] = piece(j);
        if (j < chunks && lane == 31) last[a] = piece(j + 1);
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int j = j0 + 32 * a + lane;
        uint4 b;  // (the lane behind the last chunk has what is left of the row)
        b.x = __shfl_down_sync(0xffffffffu, v[a].x, 1);
        b.y = __shfl_down_sync(0xffffffffu, v[a].y, 1);
        b.z = __shfl_down_sync(0xffffffffu, v[a].z, 1);
        b.w = __shfl_down_sync(0xffffffffu, v[a].w, 1);
        if (lane == 31) b = last[a];
        if (j + 1 == chunks) b = piece(j + 1);
        const uint32_t in[8] = {v[a].x, v[a].y, v[a].z, v[a].w,
                                b.x,    b.y,    b.z,    b.w};
        uint32_t s[6], w[5];
#pragma unroll
        for (int i = 0; i < 6; ++i) s[i] = two ? in[i + 2] : in[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = one ? s[i + 1] : s[i];
        if (j < chunks)
          *reinterpret_cast<uint4*>(out + 8 * j) =
              make_uint4(__funnelshift_r(w[0], w[1], bits),
                         __funnelshift_r(w[1], w[2], bits),
                         __funnelshift_r(w[2], w[3], bits),
                         __funnelshift_r(w[3], w[4], bits));
      }
    }
  }
}

// dW's rows to where they belong, on any 2-byte boundary: the other way round.
// A warp writes a row in aligned 16-byte pieces, each from its lane's chunk and
// the one before; a piece that lies partly outside the row as single elements.
// (Written by the products' epilogue instead, two or four bytes a lane: lay_out.)
__global__ void __launch_bounds__(1024)
    unpack_dw_kernel(const __grid_constant__ VocabCall p) {
  griddep_wait();
  griddep_launch_dependents();
  if (p.header->dw_splits > 1) return;  // (finish_grad_kernel has written it)
  constexpr int kAhead = 4;
  const int lane = threadIdx.x & 31, n = p.D, chunks = (n + 7) / 8;
  const long long extent = 2 * ((p.V - 1) * p.lddw + n);
  for (long long r = blockIdx.x * 32ll + (threadIdx.x >> 5); r < p.V;
       r += gridDim.x * 32ll) {
    const uint4* from = reinterpret_cast<const uint4*>(
        static_cast<const uint16_t*>(p.dWp) + r * p.ldxp);
    uint16_t* row = static_cast<uint16_t*>(p.dW) + r * p.lddw;
    const int off = (reinterpret_cast<uintptr_t>(row) & 15u) >> 1;
    const int start = (8 - off) & 7;  // in the chunk before
    const bool two = start & 4, one = start & 2;
    const int bits = (start & 1) * 16;
    const int pieces = (n + off + 7) / 8;
    for (int j0 = 0; j0 < pieces; j0 += 32 * kAhead) {
      uint4 v[kAhead], first[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int j = j0 + 32 * a + lane;
        v[a] = first[a] = make_uint4(0, 0, 0, 0);
        if (j < chunks) v[a] = from[j];
        if (lane == 0 && j > 0 && j - 1 < chunks) first[a] = from[j - 1];
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int j = j0 + 32 * a + lane, e = 8 * j - off;
        uint4 b;
        b.x = __shfl_up_sync(0xffffffffu, v[a].x, 1);
        b.y = __shfl_up_sync(0xffffffffu, v[a].y, 1);
        b.z = __shfl_up_sync(0xffffffffu, v[a].z, 1);
        b.w = __shfl_up_sync(0xffffffffu, v[a].w, 1);
        if (lane == 0) b = first[a];
        const uint32_t in[8] = {b.x,    b.y,    b.z,    b.w,
                                v[a].x, v[a].y, v[a].z, v[a].w};
        uint32_t s[6], w[5];
#pragma unroll
        for (int i = 0; i < 6; ++i) s[i] = two ? in[i + 2] : in[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = one ? s[i + 1] : s[i];
        uint4 o = make_uint4(__funnelshift_r(w[0], w[1], bits),
                             __funnelshift_r(w[1], w[2], bits),
                             __funnelshift_r(w[2], w[3], bits),
                             __funnelshift_r(w[3], w[4], bits));
        if (off == 0) o = v[a];
        if (j >= pieces) continue;
        if (e >= 0 && e + 8 <= n) {
          if (span_ok(row + e, 16, p.dW, extent, p.status))
            *reinterpret_cast<uint4*>(row + e) = o;
          continue;
        }
        const uint32_t q[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (e + i >= 0 && e + i < n &&
              span_ok(row + e + i, 2, p.dW, extent, p.status))
            row[e + i] = (uint16_t)(q[i >> 1] >> (16 * (i & 1)));
      }
    }
  }
}

// A tile's time in 64-deep steps: its own, or its epilogue's where that is
// longer (about eight steps: 8 warps make 128 × 256 outputs per CTA).
__device__ __forceinline__ int tile_cost(int steps) {
  return max(steps, 8) + 1;
}

// Slots that dW's tiles are summed in: 1 unless so few tiles are left to
// the pairs that one tile's depth outlasts an even share by a quarter.
__device__ __forceinline__ int dw_splits(const VocabCall& p, int rows,
                                         int pairs) {
  const int wide = vocab_tiles(p.D), depth = vocab_steps(rows);
  const int tiles = vocab_tiles(p.piece) * wide;
  if (p.dw_max_splits < 2 || tiles >= pairs) return 1;
  const int even = (tiles * depth +
                    vocab_tiles(rows) * wide * vocab_steps(p.piece)) /
                       pairs + 1;
  if (4 * depth <= 5 * even) return 1;
  return max(1, min(min((depth + even - 1) / even, depth / kVocabLeastDwShare),
                    p.dw_max_splits));
}

// How dW and dX (of `rows` rows) are cut, by 128 threads, a pair a thread.
// Each pair's share of dX's line (VocabShare) is what its tiles of G and dW
// leave of an even total, in stretches that keep a tile's slots within the
// room for them and no share under eight steps.  The first pairs have one tile
// of dW more than the others, the last one of G; so the pairs fall into three
// runs with one room each, and everything has a closed form.  (All step counts
// are below 2^30: the host checks.)
__device__ void share_out(const VocabCall& p, int rows, int* s_end) {
  VocabHeader* h = p.header;
  const int pair = threadIdx.x, pairs = p.pairs;
  const int splits = dw_splits(p, rows, pairs);
  const int dw_wide =
      p.pieces > 1 || splits > 1
          ? kVocabTile
          : vocab_tile_width(p.V, p.D, vocab_steps(rows), 128, pairs);
  if (pair == 0) {
    h->dw_splits = splits;
    h->dw_wide = dw_wide;
    h->dx_rounds = 0;
  }
  if (rows == 0) {
    if (pair < pairs) h->share[pair] = VocabShare{0, 0, 0};
    return;
  }
  const int tiles = vocab_tiles(rows) * vocab_tiles(p.D);
  const int tall = vocab_tiles(p.piece), line = vocab_steps(p.piece);
  const int tiles_w = tall * ((p.D + dw_wide - 1) / dw_wide) * splits;
  // (G of kept logits is made outside)
  const int tiles_g =
      p.pieces > 1 && !p.logits ? vocab_tiles(rows) * tall : 0;
  const int cost_w = max(
      1, tile_cost(vocab_steps(rows) / splits) * dw_wide / kVocabTile);
  const int cost_g = tile_cost(vocab_steps(p.D));
  const int more_w = tiles_w % pairs, more_g = tiles_g % pairs;
  const int end0 = min(more_w, pairs - more_g);
  const int end1 = max(more_w, pairs - more_g);
  const unsigned c0 = more_w ? cost_w : 0, c2 = more_g ? cost_g : 0;
  const unsigned c1 = more_w > pairs - more_g ? cost_w + cost_g : 0;
  const int n0 = end0, n1 = end1 - end0, n2 = pairs - end1;
  // the level, over what every pair has, at which the room under it holds
  // all steps
  unsigned level = INT_MAX;
#pragma unroll 1
  for (int round = 0; round < 4; ++round) {
    unsigned sum = tiles * line, count = 0;
    if (n0 && c0 < level) sum += n0 * c0, count += n0;
    if (n1 && c1 < level) sum += n1 * c1, count += n1;
    if (n2 && c2 < level) sum += n2 * c2, count += n2;
    const unsigned now = (sum + count - 1) / count;
    if (now >= level) break;
    level = now;
  }
  int room0 = level > c0 ? level - c0 : 0, room1 = level > c1 ? level - c1 : 0;
  int room2 = level > c2 ? level - c2 : 0;
  // whole rounds: what the fullest pair has room for
  int least = INT_MAX;
  if (n0) least = room0;
  if (n1) least = min(least, room1);
  if (n2) least = min(least, room2);
  const int rounds = min(least / line, tiles / pairs);
  const int left = (tiles - rounds * pairs) * line;
  const long long slot = (long long)vocab_tiles(rows) * kVocabTile;
  const int most = (int)max(1ll, min(1ll << 30, p.slot_rows / max(1ll, slot)));
  const int cut =
      max((line + most - 1) / most, min(line, kVocabLeastDxShare));
  room0 -= rounds * line;
  room1 -= rounds * line;
  room2 -= rounds * line;
  // the ends of the shares
  const int q = pair + 1;
  int end = left;
  if (q < pairs) {
    const long long sum = (long long)min(q, end0) * room0 +
                          (long long)max(0, min(q, end1) - end0) * room1 +
                          (long long)max(0, q - end1) * room2;
    if (sum < left) {
      const int x = (int)sum, tile = x / line, k = x - tile * line;
      end = tile * line + min(line, (k + cut / 2) / cut * cut);
    }
  }
  s_end[q] = end;
  if (pair == 0) {
    s_end[0] = 0;
    h->dx_rounds = rounds;
  }
  asm volatile("bar.sync 1, 128;\n" ::: "memory");  // these 128 threads
  const int whole = rounds * pairs;
  for (int tile = pair; tile < whole; tile += 128) p.tile_slots[tile] = 1;
  if (pair >= pairs) return;
  VocabShare s = {s_end[pair], end, 0};
  if (s.x0 < s.x1) {
    const int first = s.x0 / line, start = first * line;
    for (int j = pair; j > 0 && s_end[j] > start; --j)
      s.slot += s_end[j] > s_end[j - 1];
    // the tiles that end with this share
    int slot = s.slot;
    for (int tile = first; (tile + 1) * line <= s.x1; ++tile, slot = 0)
      p.tile_slots[whole + tile] = slot + 1;
  }
  h->share[pair] = s;
}

// Numbers the tokens that are learnt from, in order, and packs their rows of
// X where they are not read in place (some token is not learnt from, or X
// has no tensor map); packs W's rows where they have no tensor map.  Every
// block counts all learnt tokens and those before its own share (the targets
// come from L2), and numbers that share.  Forward: loss and lse of the other
// tokens are 0.  Gradients: what brings the largest |g·τ| to 1, or 2^14 for
// binary16, and how dW and dX are cut.  Most losses are means, with one g for
// all tokens: rounded as it is, g's own error (up to 2^-8 of it in bfloat16)
// would be the same in every token's target, and stay in all sums; scaled to
// 1, the target's G is p - 1, just below a power of two, where roundings are
// least.
__global__ void __launch_bounds__(1024)
    number_tokens_kernel(const __grid_constant__ VocabCall p, int forward) {
  __shared__ int s_all[32], s_before[32], s_end[kVocabMaxPairs + 1];
  __shared__ float s_most[32];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long share = (p.T + gridDim.x - 1) / gridDim.x;
  const long long own0 = min((long long)p.T, blockIdx.x * share);
  const long long own1 = min((long long)p.T, own0 + share);
  const bool scaled = !forward && blockIdx.x == 0;
  int all = 0, before = 0;
  float most = 0.f;
#pragma unroll 8
  for (long long t = threadIdx.x; t < p.T; t += 1024) {
    const bool learnt = vocab_is_learnt(p, t);
    all += learnt;
    before += learnt && t < own0;
    // (read whether learnt or not, so that no load waits for another)
    float g = scaled ? fabsf(p.grad_loss[t * p.grad_stride]) : 0.f;
    // (p·|log p + H| is at most 1/e + H)
    if (scaled && p.grad_entropy)
      g += fabsf(p.grad_entropy[t * p.entropy_stride]) * (0.4f + p.entropy[t]);
    most = fmaxf(most, learnt ? g : 0.f);
  }
  all = __reduce_add_sync(0xffffffffu, all);
  before = __reduce_add_sync(0xffffffffu, before);
  for (int o = 16; o; o >>= 1)
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (lane == 0) {
    s_all[warp] = all;
    s_before[warp] = before;
    s_most[warp] = most;
  }
  __syncthreads();
  all = __reduce_add_sync(0xffffffffu, s_all[lane]);
  before = __reduce_add_sync(0xffffffffu, s_before[lane]);
  const bool x_fits = vocab_maps(p.X, p.ldx);
  const int lo =
      forward || p.T > kVocabFewTokens ? 0 : (all + 31) / 32 * 32;
  const bool packed = !x_fits || all != p.T || lo;
  if (all != p.T) {
    if (warp == 0)
      for (long long t0 = own0; t0 < own1; t0 += 32) {
        const long long t = t0 + lane;
        const bool learnt = t < own1 && vocab_is_learnt(p, t);
        const unsigned votes = __ballot_sync(0xffffffffu, learnt);
        const int r = before + __popc(votes & ((1u << lane) - 1u));
        before += __popc(votes);
        if (t < own1) {
          p.row[t] = learnt ? r : -1;
          if (learnt) p.token[r] = (int)t;
          if (forward && !learnt) {
            p.loss[t] = 0.f;
            p.lse_out[t] = 0.f;
            if (p.entropy_out) vocab_unscored(p, t);
          }
        }
      }
    __syncthreads();
  }
  if (lo) {  // a few rows, all threads on each, written twice
    const uint16_t* from = static_cast<const uint16_t*>(p.X);
    uint16_t* to = static_cast<uint16_t*>(p.Xp);
    const int chunks = (p.D + 7) / 8, rows = (int)(own1 - own0);
    for (int k = threadIdx.x; k < rows * chunks; k += 1024) {
      const long long t = own0 + k / chunks;
      const int c = 8 * (k % chunks), r = all != p.T ? p.row[t] : (int)t;
      if (r < 0) continue;
      const uint4 v = read_8(from + t * p.ldx, c, p.D, x_fits);
      *reinterpret_cast<uint4*>(to + r * p.ldxp + c) = v;
      *reinterpret_cast<uint4*>(to + (r + lo) * p.ldxp + c) = v;
    }
    for (int r = all + blockIdx.x; r < lo; r += gridDim.x)
      for (int c = 8 * threadIdx.x; c < p.D; c += 8192) {
        const uint4 zero = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(to + r * p.ldxp + c) = zero;
        *reinterpret_cast<uint4*>(to + (r + lo) * p.ldxp + c) = zero;
      }
  } else if (packed) {
    uint16_t* to = static_cast<uint16_t*>(p.Xp);
    pack_rows(static_cast<const uint16_t*>(p.X), p.ldx, p.D, to, p.ldxp,
              all != p.T ? p.row : nullptr, x_fits, own0 + warp, own1, 32,
              lane);
    if (blockIdx.x == 0)  // Dw sums over the rows up to a multiple of 64
      for (int r = all + warp; r < (all + 63) / 64 * 64; r += 32)
        for (int c = 8 * lane; c < p.D; c += 256)
          *reinterpret_cast<uint4*>(to + r * p.ldxp + c) =
              make_uint4(0, 0, 0, 0);
  }
  if (blockIdx.x == 0) {
    if (!forward && threadIdx.x < 128)
      share_out(p, vocab_rows(all, lo), s_end);
    if (threadIdx.x == 1023) {  // (a warp that does not share out)
      for (int w = 0; w < 31; ++w) most = fmaxf(most, s_most[w]);
      most *= p.entropy ? p.inv_tau : p.tau;
      // 0, Inf and NaN: no scale; outside 2^±100 only its power of two
      const float top = p.type == GEMM_F32_MIXED_F16 ? 16384.f : 1.f;
      float scale = 1.f, inv_scale = 1.f;
      if (scaled && most >= 0x1p-100f && most <= 0x1p100f) {
        scale = top / most;
        inv_scale = most / top;
      } else if (scaled && most > 0.f && most < INFINITY) {
        scale = most < 1.f ? 0x1p100f : 0x1p-100f;
        inv_scale = 1.f / scale;
      }
      VocabHeader* h = p.header;
      h->learnt = all;
      h->packed = packed;
      h->lo = lo;
      h->scale = scale;
      h->inv_scale = inv_scale;
      // (G is stored in blocks of 64 columns, half a tile's least)
      h->wide = all == p.T || p.pieces > 1
                    ? p.wide
                    : vocab_tile_width(all, p.V, vocab_steps(p.D),
                                       forward ? 64 : 128, p.pairs);
    }
  }
  if (p.w_packed) return;
  if (p.Wp && (p.D + 7) / 8 >= kLongRow)
    pack_long_rows(static_cast<const uint16_t*>(p.W), p.ldw, p.D,
                   static_cast<uint16_t*>(p.Wp), p.ldxp, nullptr,
                   blockIdx.x * 32 + warp, p.V, gridDim.x * 32, lane);
  else if (p.Wp)
    pack_rows(static_cast<const uint16_t*>(p.W), p.ldw, p.D,
              static_cast<uint16_t*>(p.Wp), p.ldxp, nullptr, false,
              blockIdx.x * 32 + warp, p.V, gridDim.x * 32, lane);
}

// ------------------------------------------------------------- results
__device__ __forceinline__ float2 merge_stats(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  const float ref = m == -INFINITY ? 0.f : m;
  return make_float2(m, a.y * exp2f(a.x - ref) + b.y * exp2f(b.x - ref));
}

__device__ __forceinline__ float2 merge_over(float2 st, int from) {
  for (int o = from; o < 32; o <<= 1)
    st = merge_stats(st, make_float2(__shfl_xor_sync(0xffffffffu, st.x, o),
                                     __shfl_xor_sync(0xffffffffu, st.y, o)));
  return st;
}

// loss and lse: 8 rows a block, blockDim / 8 threads a row that share out its
// statistics and join them in a fixed order.
__global__ void __launch_bounds__(1024)
    finish_loss_kernel(const __grid_constant__ VocabCall p) {
  __shared__ float2 s_part[32][8];
  griddep_wait();
  griddep_launch_dependents();
  const int r = blockIdx.x * 8 + (threadIdx.x & 7);
  const int slice = threadIdx.x >> 3, warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31, j0 = lane >> 3;
  const int learnt = p.header ? p.header->learnt : p.T;
  const int wide = p.header ? p.header->wide : p.wide;
  const int parts = (int)((2ll * p.V + wide - 1) / wide);  // half tiles
  bool here = r < learnt;
  // the first warp's later loads, ahead of the statistics'
  long long t = r;
  int id = INT_MAX;
  float lq = 0.f, at = 0.f;
  bool ignored = false;
  if (warp == 0 && here) {
    if (learnt != p.T) t = p.token[r];
    if (!p.header) ignored = !vocab_is_learnt(p, t);
    if (j0 < p.top && !ignored) {
      id = p.targets ? 0 : p.ids[t * p.top + j0];
      lq = p.targets ? 0.f : p.weights[t * p.top + j0];
      at = p.picked[(long long)r * p.top + j0];
    }
  }
  // This thread's share, with what each addition rounds off kept (`lost`):
  // 2^30 words are 65536 sums in a row, whose roundings, all one way where the
  // sums are alike, left lse wrong by 4e-4.
  float2 st = make_float2(-INFINITY, 0.f);
  float lost = 0.f;
  if (here) {
#pragma unroll 4
    for (int e = slice; e < parts; e += blockDim.x >> 3) {
      const float2 b = p.stats[(long long)e * learnt + r];
      const float m = fmaxf(st.x, b.x);
      const float ref = m == -INFINITY ? 0.f : m;
      const float keep = exp2f(st.x - ref);
      const float was = st.y * keep;
      const float more = b.y * exp2f(b.x - ref) - lost * keep;
      st = make_float2(m, was + more);
      lost = (st.y - was) - more;
    }
  }
  st = merge_over(st, 8);
  const int warps = blockDim.x >> 5;
  if (warps > 1) {
    if (lane < 8) s_part[warp][lane] = st;
    __syncthreads();
    if (warp > 0) return;
    st = make_float2(-INFINITY, 0.f);
    for (int w = j0; w < warps; w += 4)
      st = merge_stats(st, s_part[w][lane & 7]);
    st = merge_over(st, 8);
  }
  const float l = st.x * 0.69314718056f + logf(st.y);
  float sum = 0.f;
  for (int j = j0; id != INT_MAX;) {
    const float q = expf(lq);
    if (q != 0.f) sum += q * (lq - (at - l));  // 0·log 0 = 0
    j += 4;
    if (j >= p.top) break;
    id = p.ids[t * p.top + j];
    lq = p.weights[t * p.top + j];
    at = p.picked[(long long)r * p.top + j];
  }
  for (int o = 8; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (here && lane < 8) {
    p.loss[t] = ignored ? 0.f : p.tau * p.tau * sum;
    p.lse_out[t] = ignored ? 0.f : l;
  }
}

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// The sum of n slots, `next` apart, in order; in two parts, with those `second`
// behind them.
template <int AHEAD, int PARTS>
__device__ __forceinline__ float4 sum_slots(const float* from, long long next,
                                            int n, long long second = 0) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int s0 = 0; s0 < n; s0 += AHEAD) {
    float4 a[AHEAD][PARTS];
#pragma unroll
    for (int s = 0; s < AHEAD; ++s)  // (past the end, the last again)
#pragma unroll
      for (int part = 0; part < PARTS; ++part)
        a[s][part] = *reinterpret_cast<const float4*>(
            from + min(s0 + s, n - 1) * next + part * second);
#pragma unroll
    for (int s = 0; s < AHEAD; ++s)
#pragma unroll
      for (int part = 0; part < PARTS; ++part)
        if (s0 + s < n) v = add4(v, a[s][part]);
  }
  return v;
}

__device__ __forceinline__ void store16(__nv_bfloat16* p, float v) {
  *p = __float2bfloat16_rn(v);
}
__device__ __forceinline__ void store16(__half* p, float v) {
  *p = __float2half_rn(v);
}

// (to: column i of a row of n, in a matrix at `base` of `rows` rows)
template <typename T16>
__device__ __forceinline__ void store_4(T16* to, float4 v, float scale, int i,
                                        int n, const void* base,
                                        long long rows, long long ld,
                                        unsigned int* status) {
  if (!span_ok(to, 2 * min(4, n - i), base, 2 * ((rows - 1) * ld + n), status))
    return;
  T16 o[4];
  store16(o, v.x * scale);
  store16(o + 1, v.y * scale);
  store16(o + 2, v.z * scale);
  store16(o + 3, v.w * scale);
  if (i + 4 <= n && (reinterpret_cast<uintptr_t>(to) & 7u) == 0) {
    *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(o);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (i + j < n) to[j] = o[j];
}

// dX, four columns a thread at a time: the sum of its tiles' slots in order,
// rounded; zeros for the tokens that are not learnt from.  And dW where its
// tiles were summed in slots.  AHEAD slots are read side by side: many where
// there are few elements, whose tiles are cut finely (they were one row of
// tiles), few otherwise.
// PARTS: of G, and so of dX.
template <typename T16, int AHEAD, int PARTS>
__global__ void __launch_bounds__(256)
    finish_grad_kernel(const __grid_constant__ VocabCall p) {
  griddep_wait();
  griddep_launch_dependents();
  const VocabHeader* h = p.header;
  const int learnt = h->learnt, wide = vocab_tiles(p.D);
  const float inv_scale = h->inv_scale;
  const long long next =
      (long long)vocab_tiles(learnt) * kVocabTile * p.ld_slot;
  const int chunks = (int)(p.ld_slot / 4);
  const long long stride = gridDim.x * 256ll;
  const long long first = blockIdx.x * 256ll + threadIdx.x;
  for (long long k = first; k < (long long)p.T * chunks; k += stride) {
    const long long t = k / chunks;
    const int i = (int)(k - t * chunks) * 4;
    const int r = learnt == p.T ? (int)t : p.row[t];
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r >= 0) {
      // this tile's place in the order of the walk (tile_coords)
      const int tm = r / kVocabTile, group = tm / kVocabGroup * kVocabGroup;
      const int high = min(vocab_tiles(learnt) - group, kVocabGroup);
      const int n =
          p.tile_slots[group * wide + i / kVocabTile * high + (tm - group)];
      // (both parts lie in one row of tiles)
      v = sum_slots<AHEAD, PARTS>(p.slots + (long long)r * p.ld_slot + i, next,
                                  n, PARTS > 1 ? h->lo * p.ld_slot : 0);
    }
    store_4(static_cast<T16*>(p.dX) + t * p.lddx + i, v, inv_scale, i, p.D,
            p.dX, p.T, p.lddx, p.status);
  }
  const int splits = h->dw_splits;
  if (splits == 1) return;
  // one piece: the whole of dW (its slots' rows are ld_slot apart)
  for (long long k = first; k < (long long)p.V * chunks; k += stride) {
    const long long r = k / chunks;
    const int i = (int)(k - r * chunks) * 4;
    const float4 v = sum_slots<AHEAD, 1>(
        p.dw_slots + 4 * k, (long long)p.dw_slot_rows * p.ld_slot, splits);
    store_4(static_cast<T16*>(p.dW) + r * p.lddw + i, v, inv_scale, i, p.D,
            p.dW, p.V, p.lddw, p.status);
  }
}

// ------------------------------------------------------------- host side
int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Places a call's state in its workspace (c.token .. c.dw_max_splits), from
// T, V, D, top and what follows them alone; returns its bytes.  The pointers
// are offsets from `ws` and only numbers where it is null.  alternatives: of
// log probabilities (-1: of a loss), whose logits are kept or not.  aligned: W
// has a tensor map (else there is room for its packed copy, unless that is kept).
int64_t lay_out(VocabCall* c, char* ws, int64_t T, int64_t V, int64_t D,
                int64_t top, bool grad, bool aligned, int64_t alternatives = -1,
                bool keep = false) {
  const bool pack_w = !aligned && !keep;
  // dW of such a width, one row behind the other, has no tensor map either.  One
  // row of tiles waits for memory: it writes dW in rows that have one, which
  // are then moved.  Short rows cost the move more, and more tokens' products
  // hide what the epilogue takes.  Gradients of 16 tokens, 50000 words, moved
  // and not: width 129 86 and 79 us, 201 95 and 91, 257 98 and 100, 401 114 and
  // 121, 1001 180 and 195, 2045 309 and 337; of 256 tokens: 201 88 and 88, 257 99
  // and 98, 401 117 and 119, 2045 325 and 345; of 300 tokens 120 and 116 at 257,
  // 141 and 136 at 401, 215 and 220 at 1001, 384 and 400 at 2045; of 600 never
  // less (498 and 480 at 2045).  8000 words: the same bounds, but for 256 tokens
  // of widths 401 to 1501 (3 us, up to 7 %, lost).
  const bool odd_rows =
      !aligned && D % 8 != 0 && D >= 256 && T <= kVocabTile;
  // A piece's G: small enough that it and its part of W stay near the L2
  // they are read from again (1800 learnt tokens of 6000, 65537 × 2048: 32,
  // 64, 128, 256 MB 1560, 1400, 1350, 1500 us a step), large enough that a
  // launch's ends do not count (4096 × 128000 × 4096: within 2 % from 64 MB
  // on).  Two are held where there are more.  dX's slots: six of an
  // 8192 × 4096 dX, or more of a smaller one.
  constexpr int64_t kMostG = 128ll << 20;
  constexpr int64_t kMostSlots = 768ll << 20;
  constexpr int64_t kMostDwSlots = 128ll << 20;
  // Logits of which the largest are looked for: those of as many tokens (but
  // 256 at least) are stored at a time.  (Each time is a launch, with its ends,
  // and reads W again: 8192 × 100000 × 2048, one word each: 2560 us with 1 GB
  // at a time, 2533 with 4.)
  constexpr int64_t kMostLogits = 4ll << 30;
  const int64_t rows = std::max<int64_t>(T, 1);
  int64_t at = 0;
  auto take = [&](auto** to, int64_t bytes) {
    *to = reinterpret_cast<std::remove_reference_t<decltype(**to)>*>(
        reinterpret_cast<uintptr_t>(ws) + at);
    at += up(bytes, 256);
  };
  take(&c->header, sizeof(VocabHeader));
  take(&c->token, rows * 4);
  take(&c->row, rows * 4);
  take(&c->learnt_flag, rows);
  take(&c->ids, rows * top * 4);
  take(&c->weights, rows * top * 4);
  c->blocks = (int)((V + 127) / 128);
  take(&c->starts, alternatives < 0 ? rows * c->blocks * 4 : 0);
  c->ldxp = up(D, 8);
  char* bytes = nullptr;
  c->xp_rows = grad && T <= kVocabFewTokens ? 2 * up(rows, 32) : up(rows, 64);
  take(&bytes, c->xp_rows * c->ldxp * 2);
  c->Xp = bytes;
  c->Wp = nullptr;
  if (pack_w) {
    take(&bytes, V * c->ldxp * 2);
    c->Wp = bytes;
  }
  if (!grad) {
    c->pieces = 1;
    // one for each row of a half tile: 128 columns, or down to 32 where two
    // rounds of 256 × 256 tiles hold all logits
    const int64_t narrow = std::min<int64_t>(
        (V + 31) / 32 * rows, 2 * kVocabMaxPairs * 8 * kVocabTile);
    const int64_t halves = std::max((V + 127) / 128 * rows, narrow);
    if (alternatives < 0) take(&c->stats, halves * 8);
    take(&c->picked, rows * top * 4);
    if (alternatives < 0) return at;
    take(&c->sums, halves * 16);
    c->chunk = (int)rows;
    c->ld_logits = up(V, 8);
    if (alternatives > 0 && !keep) {
      c->chunk = (int)std::min<int64_t>(
          rows, std::max<int64_t>(
                    kVocabTile, kMostLogits / (4 * c->ld_logits) /
                                    kVocabTile * kVocabTile));
      take(&c->logits, c->chunk * c->ld_logits * 4);
    }
    return at;
  }
  take(&c->terms, alternatives < 0 ? 0 : rows * 16);
  take(&c->goals, alternatives < 0 ? 0 : rows * 4);
  // equal pieces, whole tiles, of at most kMostG bytes of G
  const int64_t g_rows = up(rows, kVocabTile);
  const int64_t widest = std::max<int64_t>(
      kVocabTile, kMostG / (2 * g_rows) / kVocabTile * kVocabTile);
  int64_t pieces = (V + widest - 1) / widest;
  const int64_t piece = up((V + pieces - 1) / pieces, kVocabTile);
  pieces = (V + piece - 1) / piece;
  c->piece = (int)piece, c->pieces = (int)pieces;
  c->g_rows = (int)g_rows;
  take(&bytes, (pieces > 1 ? 2 : 1) * g_rows * piece * 2);
  c->G = bytes;
  take(&c->tile_slots, (int64_t)vocab_tiles(rows) * vocab_tiles(D) * 4);
  c->ld_slot = up(D, 4);
  const int64_t slot = g_rows * c->ld_slot * 4;
  // (as many as pairs, or as a tile's steps give shares)
  const int64_t line = vocab_steps(piece);
  const int64_t least = std::min<int64_t>(line, kVocabLeastDxShare);
  const int64_t shares =
      std::min<int64_t>(kVocabMaxPairs, (line + least - 1) / least);
  c->slot_rows =
      g_rows * std::min(shares, std::max<int64_t>(1, kMostSlots / slot));
  take(&c->slots, c->slot_rows * c->ld_slot * 4);
  // dW's slots: only where the whole vocabulary is one piece of few tiles
  c->dw_slot_rows = (int)up(V, 32);
  c->dw_max_splits = 1;
  c->dw_slots = nullptr;
  if (pieces == 1 &&
      (int64_t)vocab_tiles(V) * vocab_tiles(D) < kVocabMaxPairs)
    c->dw_max_splits = (int)std::max<int64_t>(
        1, std::min<int64_t>(
               {kVocabMaxDwSplits, vocab_steps(T) / kVocabLeastDwShare,
                kMostDwSlots / (c->dw_slot_rows * c->ld_slot * 4)}));
  if (c->dw_max_splits > 1)
    take(&c->dw_slots, c->dw_max_splits * c->dw_slot_rows * c->ld_slot * 4);
  c->dWp = nullptr;
  if (odd_rows) {
    take(&bytes, V * c->ldxp * 2);
    c->dWp = bytes;
  }
  return at;
}

// A call as the entry points give it.
struct Request {
  int type;
  int64_t T, V, D;
  const void* X;
  int64_t ldx;
  const void* W;
  int64_t ldw;
  bool distill;
  const int64_t* targets;
  int64_t top;
  const float* top_logits;
  int64_t ldt;
  const int64_t* top_ids;
  int64_t ldi;
  float tau;
  bool grad;
  float *loss, *lse_out;
  const float *lse, *grad_loss;
  int64_t grad_stride;
  void* dX;
  int64_t lddx;
  void* dW;
  int64_t lddw;
  // log probabilities
  bool score;
  float *entropy_out, *top_logp;
  int64_t* top_out;
  int64_t alternatives;
  void* kept;
  int64_t kept_bytes;
  const float *entropy, *grad_entropy;
  int64_t entropy_stride;
  void* ws;
  int64_t ws_bytes;
  gemm_f32_stream_t stream;
};

// Sizes (none negative) that the kernels and the workspace's bytes can count.
bool countable(int64_t T, int64_t V, int64_t D) {
  return T <= kVocabMost && V <= kVocabMost && D <= kVocabMost &&
         T * D <= kVocabMostElements && V * D <= kVocabMostElements;
}

bool logits_countable(int64_t T, int64_t V) {
  return vocab_tiles(T) * (V / kVocabTile + 1) <= 1 << 30;
}

// Bytes of the kept logits, whole rows on 32-byte boundaries with two numbers
// more each, and of W's packed copy behind them.
int64_t kept_ld(int64_t V) { return up(V + 2, 8); }
int64_t kept_logits(int64_t T, int64_t V) {
  return up(T * kept_ld(V) * 4, 256);
}
int64_t kept_bytes(int64_t T, int64_t V, int64_t D, bool pack_w) {
  return kept_logits(T, V) + (pack_w ? V * up(D, 8) * 2 : 0);
}

// What log probabilities are given besides.
int check_score(const Request& r) {
  if (r.kept_bytes < 0 || (reinterpret_cast<uintptr_t>(r.kept) & 15u) != 0)
    return GEMM_F32_ERR_INVALID_ARG;
  if (r.alternatives < 0 || r.alternatives > kVocabMaxTop ||
      r.alternatives > r.V || r.entropy_stride < 0)
    return GEMM_F32_ERR_INVALID_ARG;
  if (r.T == 0) return GEMM_F32_OK;
  if (r.grad ? (!r.entropy || !r.kept) : !r.entropy_out)
    return GEMM_F32_ERR_INVALID_ARG;
  if (r.alternatives > 0 && (!r.top_logp || !r.top_out))
    return GEMM_F32_ERR_INVALID_ARG;
  return GEMM_F32_OK;
}

int check(const Request& r) {
  if (r.type != GEMM_F32_MIXED_BF16 && r.type != GEMM_F32_MIXED_F16)
    return GEMM_F32_ERR_INVALID_ARG;
  if (r.T < 0 || r.V < 1 || r.D < 1 || r.ldx < r.D || r.ldw < r.D)
    return GEMM_F32_ERR_INVALID_ARG;
  if (r.top < 1 || r.top > kVocabMaxTop) return GEMM_F32_ERR_INVALID_ARG;
  if (!(r.tau > 0.f) || !std::isfinite(r.tau) || !std::isfinite(1.f / r.tau))
    return GEMM_F32_ERR_INVALID_ARG;
  if (r.distill && (r.ldt < r.top || r.ldi < r.top))
    return GEMM_F32_ERR_INVALID_ARG;
  if (r.ws_bytes < 0) return GEMM_F32_ERR_INVALID_ARG;
  if (!r.W || (r.grad && !r.dW)) return GEMM_F32_ERR_INVALID_ARG;
  if (r.grad && (r.lddx < r.D || r.lddw < r.D || r.grad_stride < 0))
    return GEMM_F32_ERR_INVALID_ARG;
  if (r.T > 0) {
    if (!r.X) return GEMM_F32_ERR_INVALID_ARG;
    if (r.distill ? (!r.top_logits || !r.top_ids) : !r.targets)
      return GEMM_F32_ERR_INVALID_ARG;
    if (r.grad ? (!r.lse || !r.grad_loss || !r.dX) : (!r.loss || !r.lse_out))
      return GEMM_F32_ERR_INVALID_ARG;
  }
  if (r.score) {
    const int st = check_score(r);
    if (st != GEMM_F32_OK) return st;
  }
  if (!countable(r.T, r.V, r.D)) return GEMM_F32_ERR_UNSUPPORTED;
  if (r.kept && (!logits_countable(r.T, r.V)))
    return GEMM_F32_ERR_UNSUPPORTED;
  if (r.kept &&
      r.kept_bytes < kept_bytes(r.T, r.V, r.D, !vocab_maps(r.W, r.ldw)))
    return GEMM_F32_ERR_INVALID_ARG;
  return GEMM_F32_OK;
}

// Tiles, and the steps of a piece's products, are counted in 32 bits.
bool tiles_countable(const VocabCall& c, const Request& r) {
  const int64_t most = 1 << 30;
  const int64_t rows = vocab_tiles(r.T), wide = vocab_tiles(r.D);
  if (!logits_countable(r.T, r.V)) return false;
  if (!r.grad) return true;
  const int64_t tall = vocab_tiles(c.piece), line = vocab_steps(c.piece);
  return rows * wide * line <= most && tall * wide * vocab_steps(r.T) <= most &&
         2 * (int64_t)c.g_rows <= most && c.slot_rows <= most;
}

cudaError_t launch_targets(const VocabCall& c, bool forward, int sms,
                           cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (!c.targets) {
    int wide = 1;
    while (wide < c.top && wide < 32) wide <<= 1;
    const int tokens = kTeacherWarps * (32 / wide);  // of a block
    e = launch_pdl(teacher_kernel, dim3((c.T + tokens - 1) / tokens),
                   dim3(32 * kTeacherWarps), 0, stream, c, forward ? 1 : 0);
  }
  if (e != cudaSuccess || !c.header) return e;
  // (a block packs the rows of 32 tokens, or of 2 where there are few)
  const bool few = !forward && c.T <= kVocabFewTokens;
  const int blocks =
      c.Wp && !c.w_packed
          ? sms
          : std::min(sms, few ? (c.T + 1) / 2 : (c.T + 31) / 32);
  return launch_pdl(number_tokens_kernel, dim3(blocks), dim3(1024), 0, stream,
                    c, forward ? 1 : 0);
}

cudaError_t run_forward(VocabCall& c, int sms, const WaitCfg& wc,
                        cudaStream_t stream) {
  // One row of tiles takes its time whichever of its tokens are learnt from
  // (a row's statistics are its own): nothing is numbered, the results skip
  // the others.
  // (Kept logits have a row for each that is learnt from.)
  const bool score = c.entropy_out != nullptr;
  if (c.T <= kVocabTile && !c.Wp && vocab_maps(c.X, c.ldx) && !c.keep)
    c.header = nullptr;
  cudaError_t e = launch_targets(c, true, sms, stream);
  if (score) {
    for (int phase = 0; e == cudaSuccess && phase * (int64_t)c.chunk < c.T;
         ++phase) {
      e = vocab_score(c, wc, phase, stream);
      if (e == cudaSuccess) e = vocab_score_results(c, phase, sms, stream);
    }
    return e;
  }
  if (e == cudaSuccess) e = vocab_forward(c, wc, stream);
  if (e != cudaSuccess) return e;
  // a thread's share of a row: a few statistics
  const int parts = (c.V + 127) / 128;
  const int threads = parts <= 16 ? 32 : parts <= 128 ? 256 : 1024;
  return launch_pdl(finish_loss_kernel, dim3((c.T + 7) / 8), dim3(threads), 0,
                    stream, c);
}

cudaError_t run_gradients(const VocabCall& c, int sms, const WaitCfg& wc,
                          cudaStream_t stream) {
  cudaError_t e = launch_targets(c, false, sms, stream);
  if (e == cudaSuccess) e = vocab_gradients(c, wc, stream);
  if (e != cudaSuccess) return e;
  const int64_t chunks =
      c.ld_slot / 4 * std::max<int64_t>(c.T, c.dw_slots ? c.V : 0);
  const unsigned blocks =
      (unsigned)std::min<int64_t>((chunks + 255) / 256, 8ll * sms);
  auto launch = [&](auto* fn) {
    return launch_pdl(fn, dim3(blocks), dim3(256), 0, stream, c);
  };
  using Bf16 = __nv_bfloat16;
  const bool bf16 = c.type == GEMM_F32_MIXED_BF16;
  if (c.T <= kVocabFewTokens)
    e = bf16 ? launch(finish_grad_kernel<Bf16, 12, 2>)
             : launch(finish_grad_kernel<__half, 12, 2>);
  else if (c.T <= kVocabTile)
    e = bf16 ? launch(finish_grad_kernel<Bf16, 16, 1>)
             : launch(finish_grad_kernel<__half, 16, 1>);
  else
    e = bf16 ? launch(finish_grad_kernel<Bf16, 4, 1>)
             : launch(finish_grad_kernel<__half, 4, 1>);
  if (e != cudaSuccess || !c.dWp) return e;
  return launch_pdl(unpack_dw_kernel,
                    dim3((unsigned)std::min<int64_t>(2 * sms, (c.V + 31) / 32)),
                    dim3(1024), 0, stream, c);
}

int run(const Request& r) {
  int st = check(r);
  if (st != GEMM_F32_OK) return st;
  if (r.T == 0 && !r.grad) return GEMM_F32_OK;
  VocabCall c = {};
  const int64_t need =
      lay_out(&c, static_cast<char*>(r.ws), r.T, r.V, r.D, r.top, r.grad,
              vocab_maps(r.W, r.ldw), r.score ? r.alternatives : -1,
              r.kept != nullptr);
  if (!r.ws || (reinterpret_cast<uintptr_t>(r.ws) & 15u) != 0 ||
      r.ws_bytes < need)
    return GEMM_F32_ERR_INVALID_ARG;
  if (!tiles_countable(c, r)) return GEMM_F32_ERR_UNSUPPORTED;
  int sms = 0, cc = 0;
  WaitCfg wc;
  cudaError_t e = device_facts(&sms, &cc, &wc);
  if (e != cudaSuccess) return record_cuda_error(e);
  if (cc != 10) return GEMM_F32_ERR_UNSUPPORTED;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(r.stream);
  if (r.T == 0) {  // gradients of nothing
    e = cudaMemset2DAsync(r.dW, r.lddw * 2, 0, r.D * 2, r.V, stream);
    return e == cudaSuccess ? GEMM_F32_OK : record_cuda_error(e);
  }
  c.type = r.type;
  c.T = (int)r.T, c.V = (int)r.V, c.D = (int)r.D;
  c.X = r.X, c.ldx = r.ldx;
  c.W = r.W, c.ldw = r.ldw;
  c.tau = r.tau, c.inv_tau = 1.f / r.tau;
  c.targets = r.distill ? nullptr : r.targets;
  c.top = (int)r.top;
  c.top_logits = r.top_logits, c.ldt = r.ldt;
  c.top_ids = r.top_ids, c.ldi = r.ldi;
  c.loss = r.loss, c.lse_out = r.lse_out;
  c.lse = r.lse;
  c.grad_loss = r.grad_loss, c.grad_stride = r.grad_stride;
  c.dX = r.dX, c.lddx = r.lddx;
  c.dW = r.dW, c.lddw = r.lddw;
  if (r.kept) {
    c.logits = static_cast<float*>(r.kept);
    c.ld_logits = kept_ld(r.V);
    c.chunk = c.T;
    c.keep = 1;
    if (!vocab_maps(r.W, r.ldw)) {
      c.Wp = static_cast<char*>(r.kept) + kept_logits(r.T, r.V);
      c.w_packed = r.grad;
    }
  }
  c.entropy_out = r.entropy_out;
  c.top_logp = r.top_logp, c.top_out = r.top_out;
  c.alternatives = (int)r.alternatives;
  c.entropy = r.entropy, c.grad_entropy = r.grad_entropy;
  c.entropy_stride = r.entropy_stride;
  if (vocab_maps(r.dW, r.lddw)) c.dWp = nullptr;
  c.pairs = vocab_pairs(sms);
  c.status = wc.status;
  c.wide = c.pieces > 1 ? kVocabTile
                        : vocab_tile_width(c.T, c.V, vocab_steps(c.D),
                                           r.grad ? 128 : 64, c.pairs);
  e = r.grad ? run_gradients(c, sms, wc, stream)
             : run_forward(c, sms, wc, stream);
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
  Request c = {};
  c.type = type, c.T = T, c.V = V, c.D = D;
  c.X = X, c.ldx = ldx, c.W = W, c.ldw = ldw;
  c.targets = targets, c.top = 1, c.tau = 1.f;
  c.loss = loss, c.lse_out = lse;
  c.ws = workspace, c.ws_bytes = workspace_bytes;
  c.stream = stream;
  return run(c);
}

int gemm_f32_vocab_ce_grad(int type, int64_t T, int64_t V, int64_t D,
                           const void* X, int64_t ldx, const void* W,
                           int64_t ldw, const int64_t* targets,
                           const float* lse, const float* grad_loss,
                           int64_t grad_stride, void* dX, int64_t lddx,
                           void* dW, int64_t lddw, void* workspace,
                           int64_t workspace_bytes,
                           gemm_f32_stream_t stream) {
  Request c = {};
  c.type = type, c.T = T, c.V = V, c.D = D;
  c.X = X, c.ldx = ldx, c.W = W, c.ldw = ldw;
  c.targets = targets, c.top = 1, c.tau = 1.f;
  c.grad = true, c.lse = lse, c.grad_loss = grad_loss, c.grad_stride = grad_stride;
  c.dX = dX, c.lddx = lddx, c.dW = dW, c.lddw = lddw;
  c.ws = workspace, c.ws_bytes = workspace_bytes;
  c.stream = stream;
  return run(c);
}

int gemm_f32_vocab_distill(int type, int64_t T, int64_t V, int64_t D,
                           const void* X, int64_t ldx, const void* W,
                           int64_t ldw, int64_t top, const float* top_logits,
                           int64_t ldt, const int64_t* top_ids, int64_t ldi,
                           float temperature, float* loss, float* lse,
                           void* workspace, int64_t workspace_bytes,
                           gemm_f32_stream_t stream) {
  Request c = {};
  c.type = type, c.T = T, c.V = V, c.D = D;
  c.X = X, c.ldx = ldx, c.W = W, c.ldw = ldw;
  c.distill = true, c.top = top, c.top_logits = top_logits, c.ldt = ldt;
  c.top_ids = top_ids, c.ldi = ldi, c.tau = temperature;
  c.loss = loss, c.lse_out = lse;
  c.ws = workspace, c.ws_bytes = workspace_bytes;
  c.stream = stream;
  return run(c);
}

int gemm_f32_vocab_distill_grad(
    int type, int64_t T, int64_t V, int64_t D, const void* X, int64_t ldx,
    const void* W, int64_t ldw, int64_t top, const float* top_logits,
    int64_t ldt, const int64_t* top_ids, int64_t ldi, float temperature,
    const float* lse, const float* grad_loss, int64_t grad_stride, void* dX,
    int64_t lddx, void* dW, int64_t lddw, void* workspace,
    int64_t workspace_bytes, gemm_f32_stream_t stream) {
  Request c = {};
  c.type = type, c.T = T, c.V = V, c.D = D;
  c.X = X, c.ldx = ldx, c.W = W, c.ldw = ldw;
  c.distill = true, c.top = top, c.top_logits = top_logits, c.ldt = ldt;
  c.top_ids = top_ids, c.ldi = ldi, c.tau = temperature;
  c.grad = true, c.lse = lse, c.grad_loss = grad_loss, c.grad_stride = grad_stride;
  c.dX = dX, c.lddx = lddx, c.dW = dW, c.lddw = lddw;
  c.ws = workspace, c.ws_bytes = workspace_bytes;
  c.stream = stream;
  return run(c);
}

int gemm_f32_vocab_score(int type, int64_t T, int64_t V, int64_t D,
                         const void* X, int64_t ldx, const void* W, int64_t ldw,
                         const int64_t* ids, float temperature, int64_t top,
                         float* logp, float* lse, float* entropy,
                         float* top_logp, int64_t* top_ids, void* kept,
                         int64_t kept_bytes, void* workspace,
                         int64_t workspace_bytes, gemm_f32_stream_t stream) {
  Request c = {};
  c.type = type, c.T = T, c.V = V, c.D = D;
  c.X = X, c.ldx = ldx, c.W = W, c.ldw = ldw;
  c.targets = ids, c.top = 1, c.tau = temperature;
  c.loss = logp, c.lse_out = lse;
  c.score = true, c.entropy_out = entropy, c.alternatives = top;
  c.top_logp = top_logp, c.top_out = top_ids;
  c.kept = kept, c.kept_bytes = kept_bytes;
  c.ws = workspace, c.ws_bytes = workspace_bytes;
  c.stream = stream;
  return run(c);
}

int gemm_f32_vocab_score_grad(
    int type, int64_t T, int64_t V, int64_t D, const void* X, int64_t ldx,
    const void* W, int64_t ldw, const int64_t* ids, float temperature,
    const float* lse, const float* entropy, const void* kept,
    int64_t kept_bytes, const float* grad_logp, int64_t logp_stride,
    const float* grad_entropy, int64_t entropy_stride, void* dX, int64_t lddx,
    void* dW, int64_t lddw, void* workspace, int64_t workspace_bytes,
    gemm_f32_stream_t stream) {
  Request c = {};
  c.type = type, c.T = T, c.V = V, c.D = D;
  c.X = X, c.ldx = ldx, c.W = W, c.ldw = ldw;
  c.targets = ids, c.top = 1, c.tau = temperature;
  c.grad = true, c.lse = lse;
  c.grad_loss = grad_logp, c.grad_stride = logp_stride;
  c.dX = dX, c.lddx = lddx, c.dW = dW, c.lddw = lddw;
  c.score = true, c.entropy = entropy, c.grad_entropy = grad_entropy;
  c.entropy_stride = entropy_stride;
  c.kept = const_cast<void*>(kept), c.kept_bytes = kept_bytes;
  c.ws = workspace, c.ws_bytes = workspace_bytes;
  c.stream = stream;
  return run(c);
}

int64_t gemm_f32_vocab_score_kept_size(int64_t T, int64_t V, int64_t D,
                                       int aligned) {
  if (T < 0 || V < 1 || D < 1 || (aligned != 0 && aligned != 1))
    return -GEMM_F32_ERR_INVALID_ARG;
  if (!countable(T, V, D) || !logits_countable(T, V))
    return -GEMM_F32_ERR_UNSUPPORTED;
  return kept_bytes(T, V, D, aligned == 0);
}

int64_t gemm_f32_vocab_score_workspace_size(int64_t T, int64_t V, int64_t D,
                                            int64_t top, int keep, int grad,
                                            int aligned) {
  if (T < 0 || V < 1 || D < 1 || top < 0 || top > kVocabMaxTop || top > V ||
      (keep != 0 && keep != 1) || (grad != 0 && grad != 1) ||
      (aligned != 0 && aligned != 1))
    return -GEMM_F32_ERR_INVALID_ARG;
  if (!countable(T, V, D)) return -GEMM_F32_ERR_UNSUPPORTED;
  VocabCall c = {};
  int64_t n =
      lay_out(&c, nullptr, T, V, D, 1, false, aligned != 0, top, keep != 0);
  if (grad)  // (room for either call; W's copy is in `kept`)
    n = std::max(n,
                 lay_out(&c, nullptr, T, V, D, 1, true, aligned != 0, 0, true));
  return n;
}

int64_t gemm_f32_vocab_workspace_size(int64_t T, int64_t V, int64_t D,
                                      int64_t top, int grad, int aligned) {
  if (T < 0 || V < 1 || D < 1 || top < 1 || top > kVocabMaxTop ||
      (grad != 0 && grad != 1) || (aligned != 0 && aligned != 1))
    return -GEMM_F32_ERR_INVALID_ARG;
  if (!countable(T, V, D)) return -GEMM_F32_ERR_UNSUPPORTED;
  VocabCall c = {};
  int64_t n = lay_out(&c, nullptr, T, V, D, top, false, aligned != 0);
  if (grad)  // (room for either call)
    n = std::max(n, lay_out(&c, nullptr, T, V, D, top, true, aligned != 0));
  return n;
}

}  // extern "C"
