// What the kernels of the vocabulary losses and log probabilities and their
// caller share: the call as the kernels see it, where its state lies, and the
// counts they all make.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>

#include "common.cuh"

namespace gemm_f32_impl {

constexpr int kVocabMaxTop = 256;
constexpr uint32_t kVocabNone = 0xffff;
constexpr int kVocabTile = 256;      // rows and columns of an output tile
constexpr int kVocabMaxPairs = 128;  // CTA pairs of a launch
constexpr int kVocabMaxDwSplits = 16;
// A tile of dX is cut, and dW's depth split, into shares of at least so many
// steps (where there are as many).
constexpr int kVocabLeastDxShare = 8;
constexpr int kVocabLeastDwShare = 4;
// Up to so many tokens, G is kept in two 16-bit parts, its value's rounding
// and what that leaves: rows r and lo + r of one row of tiles, with X's row
// packed in both places, so that dW adds them up and dX's are added at the
// end.  The errors of many tokens' G average out beside the rounding of the
// results; those of a few do not (a token's dX hangs on the one or few entries
// at its targets).  The rows would be empty; a step of 16 tokens, 100000 ×
// 2048 takes 346 us with it, 340 without.  (Loading X's rows twice instead, in
// boxes of 32 rows, held up the logits by 6 us.)
constexpr int kVocabFewTokens = kVocabTile / 2;
constexpr int kVocabGroup = 16;  // tile rows walked together (L2 reuse)
// The most tokens, words and columns a call may have: rows and columns are
// 32-bit numbers, and so is what lies past the last of them, up to one piece
// of the vocabulary (2^18 words at most) and a tile.
constexpr long long kVocabMost = (1ll << 31) - (1ll << 20);
// The most elements of X or W (no device holds more, and bytes of workspace
// stay far inside 64 bits).
constexpr long long kVocabMostElements = 1ll << 48;

__host__ __device__ inline int vocab_tiles(long long n) {
  return (int)((n + kVocabTile - 1) / kVocabTile);
}
__host__ __device__ inline int vocab_steps(long long n) {
  return (int)((n + 63) / 64);
}
inline int vocab_pairs(int sm_count) {
  const int pairs = sm_count / 2;
  return pairs < 1 ? 1 : pairs > kVocabMaxPairs ? kVocabMaxPairs : pairs;
}

// dX of one piece of the vocabulary is the product G·W_p.  As many whole
// rounds of its tiles as every CTA pair has time for run one tile a pair, in
// step with each other (they share operands in L2).  The 64-deep steps of
// the tiles left over, tile after tile, are shared out as one line, so that
// all pairs end together: pair i sums steps [x0, x1) of it.  A tile's shares
// go to fp32 slots of their own (the pair's first share is its tile's number
// `slot`, its others number 0); the line is cut the same way in every piece,
// so that a slot is always written by the same share.
struct VocabShare {
  int x0, x1, slot;
};

// Written by the numbering kernel, read by the later ones.
struct VocabHeader {
  int learnt;       // tokens that are learnt from
  int packed;       // X is read from its packed copy
  int lo;           // gradients: where G's second parts start, or 0
  float scale;      // gradients: G is stored times this
  float inv_scale;  // 1 / scale
  int wide;         // columns of a tile of the logits
  int dw_wide;      // columns of a tile of dW
  int dw_splits;    // > 1: dW's tiles are summed in that many fp32 slots
  int dx_rounds;    // whole rounds of dX's tiles
  VocabShare share[kVocabMaxPairs];
};

// Columns of a tile: 256, or less where there are so few tiles that more and
// narrower ones end sooner.  A 64-deep step takes about 8, 5 and 4 units for
// 256, 128 and 64 columns (below 256 the operands' loads bound it), and the
// epilogue of a tile about as long as 8 steps of it; it follows the last
// tile.
__host__ __device__ inline int vocab_tile_width(int rows, int cols, int steps,
                                                int narrowest, int pairs) {
  const int tall = vocab_tiles(rows);
  int best = kVocabTile, best_time = INT_MAX;
  if ((long long)tall * vocab_tiles(cols) > 2 * pairs) return best;
  for (int wide = 256, step = 8, last = 64; wide >= narrowest;
       wide >>= 1, step = step == 8 ? 5 : 4, last >>= 1) {
    const int rounds = (tall * ((cols + wide - 1) / wide) + pairs - 1) / pairs;
    const int one = steps * step > last ? steps * step : last;
    const int time = rounds * one + last;
    if (time < best_time) best = wide, best_time = time;
  }
  return best;
}

// One call.  Tokens that are learnt from are numbered in order: row r of the
// products' matrices is token token[r], and row[t] is r or -1.
struct VocabCall {
  int type;  // gemm_f32_mixed_type
  int T, V, D;
  const void* X;
  long long ldx;
  const void* W;
  long long ldw;
  float tau, inv_tau;
  // cross entropy: one target a token; else null
  const int64_t* targets;
  // distillation
  int top;
  const float* top_logits;
  long long ldt;
  const int64_t* top_ids;
  long long ldi;
  // forward
  float *loss, *lse_out;
  // gradients
  const float* lse;
  const float* grad_loss;
  long long grad_stride;
  void* dX;
  long long lddx;
  void* dW;
  long long lddw;

  // log probabilities (one target a token); else null
  float* entropy_out;         // forward (loss is the log probability)
  float* top_logp;            // [T][alternatives]
  int64_t* top_out;           // their ids
  int alternatives;
  const float* entropy;       // gradients (grad_loss: of the log probability)
  const float* grad_entropy;  // or null
  long long entropy_stride;

  int pairs;  // CTA pairs of the products
  int wide;   // columns of the logits' tiles if all tokens are learnt from
  unsigned int* status;  // where a bounds check reports

  // ---- workspace
  VocabHeader* header;   // null: nothing is numbered or packed, row t is
  int *token, *row;      // token t (forward, one row of tiles)
  uint8_t* learnt_flag;  // distillation: whether anything of a token counts
  int* ids;              // distillation [T][top]: entries that count, by id,
  float* weights;        // then INT_MAX; log q (forward) or q of each
  uint32_t* starts;      // distillation [T][blocks of 128 columns]: in the
  int blocks;            // low half the number of the row's first entry in
                         // the block or after it, in the high half its column
                         // in the block (kVocabNone: it is after it)
  void* Xp;              // X's packed copy: the learnt tokens' rows, then
  long long ldxp;        // zero rows up to a multiple of 64; or, few tokens,
  long long xp_rows;     // both twice (VocabHeader::lo)
  void* Wp;              // W's packed copy, or null (W has a tensor map)
  int w_packed;       // that a call before has made
  // forward
  float2* stats;  // [half tiles' columns][learnt]: (max, sum), powers of 2
  float* picked;  // [T][top]: logits / τ of the entries (log probabilities:
                  // logits)
  // log probabilities
  float4* sums;    // in place of stats, [learnt][half tiles' columns]: (max,
                   // sum, Σ e·log2 e of its terms e, the largest logit)
  float* logits;   // [chunk][ld_logits]: the logits of the learnt tokens, of
  long long ld_logits;  // all (kept for the gradients, and behind each row its
  int chunk, keep;      // reference and log S) or, for their largest, of
                        // `chunk` in turn; or null
  // gradients
  int piece, pieces;  // columns of G; the pieces of the vocabulary
  float4* terms;      // log probabilities: what G needs of each learnt row
  int* goals;         // (score_terms), and its word
  void* G;            // [2 · g_rows][piece]: two pieces' G in turn (one
                      // piece: [g_rows][piece])
  int g_rows;
  int* tile_slots;    // slots of each tile of dX, in the order of the walk
  float* slots;       // dX: [slot_rows][ld_slot]
  long long slot_rows, ld_slot;
  float* dw_slots;    // [dw_max_splits · dw_slot_rows][ld_slot], or null
  int dw_slot_rows, dw_max_splits;
  void* dWp;  // dW in rows that have a tensor map, where its own have none and
              // there is room (ldxp apart); or null
};

// The products of a call (vocab_gemm.cu): its tensor maps, made once, and
// one launch each.
cudaError_t vocab_forward(const VocabCall& c, const WaitCfg& wc,
                          cudaStream_t stream);
cudaError_t vocab_gradients(const VocabCall& c, const WaitCfg& wc,
                            cudaStream_t stream);
// Log probabilities: chunk `phase` of the tokens.
cudaError_t vocab_score(const VocabCall& c, const WaitCfg& wc, int phase,
                        cudaStream_t stream);

// What surrounds them for log probabilities (vocab_score.cu).
// The results of chunk `phase`.
cudaError_t vocab_score_results(const VocabCall& c, int phase, int sms,
                                cudaStream_t stream);
// G of a piece of the vocabulary from the kept logits.
cudaError_t vocab_score_g(const VocabCall& c, int piece, int sms,
                          cudaStream_t stream);

// Whether a tensor map can describe a 16-bit matrix.
__host__ __device__ __forceinline__ bool vocab_maps(const void* p,
                                                    long long ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0;
}
// Eight 16-bit elements from column c of n of a row, zeros past the end.
// vec: the row is 16-byte aligned; else it is read in the aligned 4-byte
// words that hold it (a word that lies partly outside the row is read as
// single elements).
__device__ __forceinline__ uint4 read_8(const uint16_t* __restrict__ src,
                                        int c, int n, bool vec) {
  if (vec && c + 8 <= n) return *reinterpret_cast<const uint4*>(src + c);
  const int odd = (reinterpret_cast<uintptr_t>(src) >> 1) & 1;
  if (c >= odd && c + 8 + odd <= n) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(src + c - odd);
    const uint32_t a = w[0], b = w[1], d = w[2], e = w[3];
    if (!odd) return make_uint4(a, b, d, e);
    return make_uint4(__funnelshift_r(a, b, 16), __funnelshift_r(b, d, 16),
                      __funnelshift_r(d, e, 16), __funnelshift_r(e, w[4], 16));
  }
  uint32_t e[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) e[j] = c + j < n ? src[c + j] : 0;
  return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16,
                    e[6] | e[7] << 16);
}
// Two values rounded to 16 bits, and what the rounding leaves of them,
// rounded too (AB_TYPE 1: bfloat16).
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
template <int AB_TYPE>
__device__ __forceinline__ uint32_t pack16_rest(float lo, float hi,
                                                uint32_t rounded) {
  if constexpr (AB_TYPE == 1) {
    return pack16<AB_TYPE>(lo - __uint_as_float(rounded << 16),
                           hi - __uint_as_float(rounded & 0xffff0000u));
  } else {
    const float2 r =
        __half22float2(*reinterpret_cast<const __half2*>(&rounded));
    return pack16<AB_TYPE>(lo - r.x, hi - r.y);
  }
}
// 2^x by the hardware's approximation (relative error about 2^-22; x = -Inf
// gives 0), the exponential of all statistics and gradients.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// The log probability of a logit z in a row of reference m and log S.
__device__ __forceinline__ float vocab_log_prob(const VocabCall& p, float z,
                                                float m, float log_sum) {
  return fmaf(0.69314718056f, fmaf(z, p.inv_tau * 1.4426950408889634f, -m),
              -log_sum);
}
// Log probabilities' G = (a·([v = y] − p) − b·p·(log p + H))/τ, of the kept
// logits z: with t = z·c − lse·log2 e, c = log2 e / τ, p = 2^t,
//   G = p·(A + B·t) + [v = y]·a,  A = −(a + b·H),  B = −b·ln 2
// (a, b: times 1/τ and the scale of G).  Of a row: −b·H, B, a, −lse·log2 e.
//   lse's rounding (1e-6 of an lse of 16) makes a factor of p.  At the word y
// itself 1 − p would be off by it, however small it is: there log p comes from
// the row's reference and sum, which lie behind its logits, as logp does, and
//   G = −a·(exp(log p) − 1) − b·p·(H + log p).
__device__ __forceinline__ float4 score_terms(const VocabCall& p, long long t) {
  const float scale = p.header->scale * p.inv_tau;
  const float a = p.grad_loss[t * p.grad_stride] * scale;
  const float b =
      p.grad_entropy ? p.grad_entropy[t * p.entropy_stride] * scale : 0.f;
  return make_float4(-b * p.entropy[t], -b * 0.69314718056f, a,
                     -p.lse[t] * 1.4426950408889634f);
}

// A warp's part of G: 1024 columns from c0 on of row r in a piece of the
// vocabulary that starts at v0 and has `cols` columns, with zeros up to `all`;
// of few tokens (lo > 0) in two parts.  here: the row is a token's.
constexpr int kVocabGRun = 1024;
template <int AB_TYPE, typename Terms>
__device__ __forceinline__ void score_g_run(const VocabCall& p, uint16_t* G,
                                            int r, int c0, int v0, int cols,
                                            int all, int lo, bool here,
                                            int lane, Terms terms_of) {
  constexpr int kRuns = kVocabGRun / 256;
  const float c2 = p.inv_tau * 1.4426950408889634f;
  const float* z = p.logits + (long long)r * p.ld_logits + v0;
  float f[kRuns][8];
#pragma unroll
  for (int i = 0; i < kRuns; ++i) {
    const int c = c0 + 256 * i + 8 * lane;
    if (here && c + 8 <= cols) {
      const float4 x = __ldcs(reinterpret_cast<const float4*>(z + c));
      const float4 y = __ldcs(reinterpret_cast<const float4*>(z + c + 4));
      f[i][0] = x.x, f[i][1] = x.y, f[i][2] = x.z, f[i][3] = x.w;
      f[i][4] = y.x, f[i][5] = y.y, f[i][6] = y.z, f[i][7] = y.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        f[i][j] = here && c + j < cols ? z[c + j] : -INFINITY;
    }
  }
  float4 of = make_float4(0.f, 0.f, 0.f, 0.f);
  int goal = -1;
  if (here) terms_of(of, goal);
  goal -= v0;
  const long long extent = 2ll * (p.pieces > 1 ? 2 : 1) * p.g_rows * p.piece;
#pragma unroll
  for (int i = 0; i < kRuns; ++i) {
    const int c = c0 + 256 * i + 8 * lane;
    if (c >= all) break;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float t = fmaf(f[i][j], c2, of.w), e = exp2_fast(t);
      // (2^-200 is 0: an infinity's product with it would not be)
      const float g = e * fmaf(of.y, fmaxf(t, -200.f), of.x - of.z);
      f[i][j] = here && c + j < cols ? g : 0.f;
    }
    if (goal >= c && goal < c + 8) {
      const float* of_row = p.logits + (long long)r * p.ld_logits + p.V;
      const float log_p = vocab_log_prob(p, z[goal], of_row[0], of_row[1]);
      const float less = expm1f(log_p);  // p - 1
      const float t = fmaxf(log_p * 1.4426950408889634f, -200.f);
      const float g = fmaf(-of.z, less, (1.f + less) * fmaf(of.y, t, of.x));
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (goal == c + j) f[i][j] = g;
    }
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = pack16<AB_TYPE>(f[i][2 * j], f[i][2 * j + 1]);
    uint16_t* to = G + (long long)r * p.piece + c;
    if (!span_ok(to, 16, p.G, extent, p.status)) continue;
    *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
    if (!lo) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = pack16_rest<AB_TYPE>(f[i][2 * j], f[i][2 * j + 1], w[j]);
    to += (long long)lo * p.piece;
    if (span_ok(to, 16, p.G, extent, p.status))
      *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// What a token that is not scored is given besides.
__device__ __forceinline__ void vocab_unscored(const VocabCall& c,
                                               long long t) {
  c.entropy_out[t] = 0.f;
  for (int j = 0; j < c.alternatives; ++j) {
    c.top_logp[t * c.alternatives + j] = 0.f;
    c.top_out[t * c.alternatives + j] = -1;
  }
}
// Rows of the gradients' products.
__device__ __forceinline__ int vocab_rows(int learnt, int lo) {
  return lo ? 2 * lo : learnt;
}
__device__ __forceinline__ bool vocab_is_learnt(const VocabCall& c,
                                                long long t) {
  if (!c.targets) return c.learnt_flag[t] != 0;
  const int64_t y = c.targets[t];
  return y >= 0 && y < c.V;
}

}  // namespace gemm_f32_impl
