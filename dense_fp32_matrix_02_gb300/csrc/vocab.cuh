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
constexpr int kVocabTile = 256;  // rows and columns of an output tile

// Written by the first kernels of a call, read by the later ones.
struct VocabHeader {
  int learnt;       // tokens that are learnt from
  int packed;       // X is read from its packed copy
  int dx_splits;    // slots that dX is summed in
  float scale;      // gradients: G is stored times this power of two
  float inv_scale;  // 1 / scale
};

// The target distributions.  Row t of ids and log_q (top entries a row)
// holds token t's entries that count, sorted by id, then INT_MAX; a weight
// is exp(log_q).  Tokens that are learnt from are numbered in order: row r
// of the products' matrices is token token[r].
struct VocabTargets {
  const VocabHeader* header;
  const int* token;
  const int* ids;
  const float* log_q;
  int top;
  float inv_tau;
};

// The products of the vocabulary losses, with what their epilogues make.
enum VocabProduct {
  kVocabStats = 0,  // logits X·Wᵀ -> per row and 128 columns: softmax
                    // statistics; the targets' logits
  kVocabGrad = 1,   // logits X·W_pᵀ of a piece -> G, 16-bit
  kVocabDx = 2,     // G·W_p, added into fp32 slots
  kVocabDw = 3      // Gᵀ·X, 16-bit: the piece's rows of dW
};

struct VocabGemm {
  int type;         // gemm_f32_mixed_type
  int T, D;
  const void* X;    // as given; valid where header->packed is 0
  long long ldx;
  const void* Xp;   // packed: rows of the learnt tokens, then zero rows up
  long long ldxp;   // to a multiple of 64
  int rows_xp;
  const void* W;    // first row of the piece
  long long ldw;
  int v0, n;        // the piece: columns v0 .. v0 + n of the logits
  VocabTargets targets;
  // kVocabStats
  float2* stats;    // [2·tiles of 256 columns][T]: (max, sum) in powers of 2
  float* picked;    // [T][top]: logits / τ of the entries
  // kVocabGrad and the products of G
  void* G;          // [T][ldg]
  long long ldg;
  const float* lse;
  const float* grad_loss;
  long long grad_stride;
  float tau;
  // kVocabDx
  float* slots;     // [max_splits][T][ld_slot]
  long long ld_slot;
  int max_splits;
  int add;          // add to the slots (else overwrite)
  // kVocabDw
  void* dW;         // first row of the piece
  long long lddw;
};

cudaError_t launch_vocab_gemm(VocabProduct product, const VocabGemm& p,
                              int sm_count, const WaitCfg& wc,
                              cudaStream_t stream);

// How many slots dX (rows × D, each element a sum over `depth`) is summed
// in by `pairs` CTA pairs: the split of the depth that ends first, counting
// rounds of 256 × 256 tiles and, for each tile, the 64-deep steps it runs
// and about six steps' time for its epilogue.
__host__ __device__ inline int vocab_dx_splits(int rows, int D, int depth,
                                               int pairs, int most) {
  const long long tiles = (long long)((rows + kVocabTile - 1) / kVocabTile) *
                          ((D + kVocabTile - 1) / kVocabTile);
  const int steps = (depth + 63) / 64;
  int best = 1;
  long long best_cost = 0;
  for (int s = 1; s <= most && (s == 1 || steps / s >= 4); ++s) {
    const long long rounds = (tiles * s + pairs - 1) / pairs;
    const long long cost = rounds * ((steps + s - 1) / s + 6);
    if (s == 1 || cost < best_cost) {
      best = s;
      best_cost = cost;
    }
  }
  return best;
}

__device__ __forceinline__ void store16(__nv_bfloat16* p, float v) {
  *p = __float2bfloat16_rn(v);
}
__device__ __forceinline__ void store16(__half* p, float v) {
  *p = __float2half_rn(v);
}

}  // namespace gemm_f32_impl
