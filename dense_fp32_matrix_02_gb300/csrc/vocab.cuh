// What the vocabulary losses' kernels share: the targets as the kernels see
// them, the state that a call keeps in its workspace, and the products'
// launch interface.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>

#include "common.cuh"

namespace gemm_f32_impl {

constexpr int kVocabMaxTop = 256;
constexpr int kVocabTile = 256;     // rows and columns of an output tile
constexpr int kVocabMaxPairs = 128;  // CTA pairs of a launch
constexpr int kVocabMaxDwSplits = 16;
constexpr int kVocabGroup = 16;  // tile rows walked together (L2 reuse)

__host__ __device__ inline int vocab_pairs(int sm_count) {
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

// Written by the first kernels of a call, read by the later ones.
struct VocabHeader {
  int learnt;       // tokens that are learnt from
  int packed;       // X is read from its packed copy
  float scale;      // gradients: G is stored times this power of two
  float inv_scale;  // 1 / scale
  int dw_splits;    // > 1: dW's tiles are summed in that many fp32 slots
  int dx_rounds;    // whole rounds of dX's tiles
  VocabShare share[kVocabMaxPairs];
};

// The target distributions.  Row t of ids and weights (top entries a row)
// holds token t's entries that count, sorted by id, then INT_MAX, and log q
// (forward) or q (gradients) of each.  Tokens that are learnt from are numbered in order: row r
// of the products' matrices is token token[r].
struct VocabTargets {
  const VocabHeader* header;
  const int* token;
  const int* ids;
  const float* weights;
  int top;
  float inv_tau;
};

__host__ __device__ inline int vocab_tiles(long long n) {
  return (int)((n + kVocabTile - 1) / kVocabTile);
}
__host__ __device__ inline int vocab_steps(long long n) {
  return (int)((n + 63) / 64);
}
// A tile's time in 64-deep steps: its own, or its epilogue's where that is
// longer (about eight steps: 8 warps make 128 × 256 outputs per CTA).
__host__ __device__ inline int vocab_tile_cost(int steps) {
  return (steps > 8 ? steps : 8) + 1;
}
// Rows between two slots of dX.
__host__ __device__ inline long long vocab_slot_rows(int learnt) {
  return (long long)vocab_tiles(learnt) * kVocabTile;
}
// Slots that dW's tiles are summed in: 1 (none: dW is written at once)
// unless so few tiles are left to the pairs that one tile's depth outlasts
// the whole piece's even share by a quarter.
__host__ __device__ inline int vocab_dw_splits(int learnt, int n, int D,
                                               int pairs, int most) {
  const long long tw = (long long)vocab_tiles(n) * vocab_tiles(D);
  const long long tx = (long long)vocab_tiles(learnt) * vocab_tiles(D);
  const long long depth = vocab_steps(learnt);
  const long long even =
      (tw * depth + tx * vocab_steps(n) + pairs - 1) / pairs + 1;
  if (4 * depth <= 5 * even || tw >= pairs) return 1;
  long long s = (depth + even - 1) / even;
  if (s > depth / 4) s = depth / 4;
  if (s > most) s = most;
  return s > 1 ? (int)s : 1;
}

// The products of the vocabulary losses, with what their epilogues make:
//   forward: logits X·Wᵀ -> per row and 128 columns the softmax statistics;
//     the targets' logits;
//   gradients, one launch: G of piece `grad` (logits made again, 16-bit) and
//     from G of piece `back` its rows of dW = Gᵀ·X and its share of
//     dX += G·W.  Either piece may be absent (n = 0).
struct VocabPiece {
  int v0, n;  // columns v0 .. v0 + n of the logits
  void* G;    // [T][ldg]
};
struct VocabGemm {
  int type;       // gemm_f32_mixed_type
  int T, V, D;
  const void* X;  // as given; read where header->packed is 0
  long long ldx;
  const void* Xp;  // packed: rows of the learnt tokens, then zero rows up
  long long ldxp;  // to a multiple of 64
  int rows_xp;
  const void* W;
  long long ldw;
  VocabTargets targets;
  // forward
  float2* stats;  // [columns / 128][T]: (max, sum) in powers of 2
  float* picked;  // [T][top]: logits / τ of the entries
  // gradients
  VocabPiece grad, back;
  int piece;      // columns of a whole piece
  int first;      // back is the first piece: dX's slots start from it
  long long ldg;
  const float* lse;
  const float* grad_loss;
  long long grad_stride;
  float tau;
  float* slots;   // dX: [slot_rows][ld_slot]
  long long slot_rows, ld_slot;
  float* dw_slots;  // [dw_max_splits · dw_slot_rows][ld_slot], or null
  long long dw_slot_rows;
  int dw_max_splits;
  void* dW;
  long long lddw;
};

cudaError_t launch_vocab_stats(const VocabGemm& p, int sm_count,
                               const WaitCfg& wc, cudaStream_t stream);
cudaError_t launch_vocab_step(const VocabGemm& p, int sm_count,
                              const WaitCfg& wc, cudaStream_t stream);

__device__ __forceinline__ void store16(__nv_bfloat16* p, float v) {
  *p = __float2bfloat16_rn(v);
}
__device__ __forceinline__ void store16(__half* p, float v) {
  *p = __float2half_rn(v);
}

}  // namespace gemm_f32_impl
