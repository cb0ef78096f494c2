// What the vocabulary losses' kernels and their caller share: the call as
// the kernels see it, where its state lies, and the counts they all make.
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
  // forward
  float2* stats;  // [half tiles' columns][learnt]: (max, sum), powers of 2
  float* picked;  // [T][top]: logits / τ of the entries
  // gradients
  int piece, pieces;  // columns of G; the pieces of the vocabulary
  void* G;            // [2 · g_rows][piece]: two pieces' G in turn (one
                      // piece: [g_rows][piece])
  int g_rows;
  int* tile_slots;    // slots of each tile of dX, in the order of the walk
  float* slots;       // dX: [slot_rows][ld_slot]
  long long slot_rows, ld_slot;
  float* dw_slots;    // [dw_max_splits · dw_slot_rows][ld_slot], or null
  int dw_slot_rows, dw_max_splits;
};

// The products of a call (vocab_gemm.cu): its tensor maps, made once, and
// one launch each.
cudaError_t vocab_forward(const VocabCall& c, const WaitCfg& wc,
                          cudaStream_t stream);
cudaError_t vocab_gradients(const VocabCall& c, const WaitCfg& wc,
                            cudaStream_t stream);

// Whether a tensor map can describe a 16-bit matrix.
__host__ __device__ __forceinline__ bool vocab_maps(const void* p,
                                                    long long ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0;
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
