// The products of the vocabulary losses (vocab_loss.cu has the formulas) on
// the 5th-generation tensor cores: one kernel whose epilogue makes what the
// losses need of each 256 × 256 tile, so that no logits are stored:
//   Stats  z = X·Wᵀ:  per row and half tile max and Σ exp, and the logits of
//          the row's targets;
//   Grad   z = X·W_pᵀ: G = g·τ·(exp(z/τ − lse) − q), rounded to 16 bits;
//   Dw     Gᵀ·X, rounded to 16 bits (or, few tiles, into fp32 slots);
//   Dx     G·W_p, added into fp32 slots.
// Log probabilities (vocab_score.cu) take Stats with a third number, for the
// entropy, and with the logits stored where they are kept or searched; their
// gradients Dw and Dx, of a G that is made from the kept logits.
// Stats is the forward launch.  The gradients take one launch per piece of
// the vocabulary and one more, each of which makes Grad of one piece beside
// Dw and Dx of the one before: they do not depend on each other, and the
// depth of Dx is cut so that every pair of CTAs ends at the same time
// (VocabShare).  One cooperative launch for everything, with grid barriers
// between the phases, was measured against this: it saves the host about
// 4 us a launch, but the phases that are not products run on 320 threads an
// SM, and nothing of a launch overlaps the one before (777 × 9973 × 521
// distillation step 124 us against 98, 2048 × 50021 × 768 forward 140
// against 124).
//
// Persistent clusters of two CTAs, one pair per two SMs, walk the tiles.  A
// pair works on one tile by tcgen05.mma.cta_group::2 (M 256, N 256, K 16):
// each CTA holds 128 rows of A and 128 columns of B in its shared memory
// (32 KB a step of 64), the tensor cores read B from both, and each CTA's
// TMEM receives its 128 rows × 256 columns of the result.  Against a tile of
// 128 × 256 per CTA this loads a third less per multiply.  Two accumulators
// of 256 columns fill TMEM, so a tile's epilogue overlaps the next tile's
// products.
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

#include <algorithm>
#include <cstring>
#include <type_traits>

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
constexpr float kLog2e = 1.4426950408889634f;
// Steps of a logit that an accumulator in tensor memory sums before the
// epilogue adds them to its own fp32 sums.  It drops bits below its last at
// every step, towards zero: 2048 to 4096 deep, the losses' error against 64
// bits was 1-3e-6 with one sum.  At 2048 × 50021 × 768 (12 steps) it is 2.1e-7,
// with 8, 4 and 2 steps a sum 1.5e-7, 1.3e-7 and 1.2e-7 at 6, 26 and 60 % more
// time.  The fewer the tokens, the less their errors average out, and one row
// of tiles waits for W anyway: it sums 8 steps, or 4 for a few tokens (one
// token, 32000 × 768, median of 24: 4.1e-7 with 16, 2.4e-7 with 8, 1.5e-7
// with 4; 21.3, 22.8 and 24.4 us.  64 tokens, 100000 × 2048: 78 us with 8, 86
// with 4).  Grad sums as Stats does, to the bit: a token learnt by heart has
// G = p - 1 at its target, all of it the difference of that logit and lse, and
// is wrong by whatever the two calls' logits differ (by 1e-4, some times G
// itself, with one sum in Grad 2048 to 4096 deep).  So the rule goes by what
// both calls see: all tokens where the forward call may number none.  Log
// probabilities (whose logits are made once) take 8 steps of any number of
// tokens: what is dropped shrinks every logit, and the entropy of flat
// distributions with it (by 1.7e-6 at 16 steps, 7.8e-7 at 8, where sums that
// round to nearest are 7.5e-7 off: 2045 × 50021 × 1000; 8192 × 32000 × 768 270 ->
// 289 us).
__device__ __forceinline__ int sum_steps(const VocabCall& p, int learnt) {
  return p.T <= 8 ? 4 : learnt <= kVocabTile || p.sums ? 8 : 16;
}

// Steps that an accumulator sums for dW and dX, whose results are rounded to
// 16 bits: what it drops over 256 steps is 1e-4 of a sum whose terms have one
// sign, half of binary16's rounding.  It grows with the depth (65536 tokens
// 4e-4, 262144 tokens 1.5e-3).
constexpr int kDeepSteps = 256;

enum Kind { kStats, kGrad, kDw, kDx };
enum Loop { kShallow, kDeep, kLogits };  // of the gradients' epilogue

template <bool STAGED>
struct Shape {
  static constexpr int kStages = STAGED ? 6 : 7;
  static constexpr int kOffStaging = kStages * kStageBytes;
  static constexpr int kOffCtl =
      kOffStaging + (STAGED ? kEpiWarps * kStagingBytes : 0);
  struct __align__(8) Control {
    uint64_t full[kStages];   // TMA of both CTAs -> MMA (first CTA's is used)
    uint64_t empty[kStages];  // MMA completion -> producers
    uint64_t acc_full[2];     // last MMA of a sum -> epilogues
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

// One arrival on a barrier of either CTA.  What it orders, the reads of
// TMEM, has completed before it (tcgen05.wait::ld); no other memory is handed
// over, so neither it nor the wait for it needs the scope of the cluster (a
// release and acquire of that scope held up every step and every tile).
__device__ __forceinline__ void mbar_arrive_pair(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];\n" ::"r"(bar)
               : "memory");
}

// Adds a block in memory (c0 innermost).
__device__ __forceinline__ void tma_add_2d(const void* tmap, uint32_t src,
                                           int c0, int c1) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group "
      "[%0, {%2, %3}], [%1];\n" ::"l"(tmap),
      "r"(src), "r"(c0), "r"(c1)
      : "memory");
}

// f[i] = f[i]·m + a for 32 values, two to an instruction.
__device__ __forceinline__ void scale_add_32(float* f, float m, float a) {
  uint64_t mm, aa;
  asm("mov.b64 %0, {%1, %1};\n" : "=l"(mm) : "f"(m));
  asm("mov.b64 %0, {%1, %1};\n" : "=l"(aa) : "f"(a));
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    uint64_t x;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(x) : "f"(f[j]), "f"(f[j + 1]));
    asm("fma.rn.f32x2 %0, %0, %1, %2;\n" : "+l"(x) : "l"(mm), "l"(aa));
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(f[j]), "=f"(f[j + 1]) : "l"(x));
  }
}

// Two values times m, rounded to 16 bits.
template <int AB_TYPE>
__device__ __forceinline__ uint32_t pack16_scaled(float lo, float hi,
                                                  float m) {
  uint64_t x, mm;
  asm("mov.b64 %0, {%1, %1};\n" : "=l"(mm) : "f"(m));
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(x) : "f"(lo), "f"(hi));
  asm("mul.rn.f32x2 %0, %0, %1;\n" : "+l"(x) : "l"(mm));
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(lo), "=f"(hi) : "l"(x));
  return pack16<AB_TYPE>(lo, hi);
}

// The sum of 32 values, two additions to an instruction, in four runs.
__device__ __forceinline__ float sum_32(const float* f) {
  uint64_t s[2];
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    uint64_t x;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(x) : "f"(f[j]), "f"(f[j + 1]));
    if (j < 4)
      s[j >> 1] = x;
    else
      asm("add.rn.f32x2 %0, %0, %1;\n" : "+l"(s[(j >> 1) & 1]) : "l"(x));
  }
  asm("add.rn.f32x2 %0, %0, %1;\n" : "+l"(s[0]) : "l"(s[1]));
  float a, b;
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(s[0]));
  return a + b;
}

// Σ f[i]·g[i] of 32 values, two to an instruction, in four runs.
__device__ __forceinline__ float dot_32(const float* f, const float* g) {
  uint64_t s[2];
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    uint64_t x, y;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(x) : "f"(f[j]), "f"(f[j + 1]));
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(y) : "f"(g[j]), "f"(g[j + 1]));
    if (j < 4)
      asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(s[j >> 1]) : "l"(x), "l"(y));
    else
      asm("fma.rn.f32x2 %0, %1, %2, %0;\n"
          : "+l"(s[(j >> 1) & 1])
          : "l"(x), "l"(y));
  }
  asm("add.rn.f32x2 %0, %0, %1;\n" : "+l"(s[0]) : "l"(s[1]));
  float a, b;
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(s[0]));
  return a + b;
}

struct Maps {
  CUtensorMap x, xp, w;     // operands, 64 × 64 boxes
  CUtensorMap logits;       // fp32, 32 × 32
  CUtensorMap g_in, g_out;  // G: 64 × 64, 64 × 32
  CUtensorMap dw;           // 64 × 32
  CUtensorMap slots, dw_slots;  // fp32, 32 × 32
};

// ------------------------------------------------------------- the walk
// One sum of a pair: a tile (or, Dx and split Dw, a share of its depth).
struct Unit {
  int kind;
  int tm, tn, wide;  // wide: the tile's columns
  int kb0, kb1;
  int slot;
};

// Division by a number known early, in four instructions: the compiler's own
// takes some 150 cycles, and what finds a warp's next tile lies between two
// epilogues, where nothing hides it (a tile of dW, 16 tokens: 5500 cycles,
// 4900 with it; that step 363 -> 350 us, 8192 × 65536 × 1024 forward 669 ->
// 664).
struct Divisor {
  unsigned d, m;
  __device__ __forceinline__ void set(int by) {
    d = by > 1 ? by : 1;
    m = 0xffffffffu / d;
  }
  // (m is at most one below 2^32 / d, so the first quotient is right or one
  // too small)
  __device__ __forceinline__ int quotient(int n, int& rest) const {
    unsigned q = __umulhi((unsigned)n, m), r = (unsigned)n - q * d;
    if (r >= d) r -= d, ++q;
    rest = (int)r;
    return (int)q;
  }
};

// The order of m × n tiles: tile_coords.
struct Tiles {
  int m;
  Divisor group;  // tiles of a group of rows
  __device__ __forceinline__ void set(int m_, int n) {
    m = m_;
    group.set(kVocabGroup * n);
  }
  __device__ __forceinline__ void coords(int j, int& tm, int& tn) const {
    int in;
    const int first = group.quotient(j, in) * kVocabGroup;
    if (first + kVocabGroup <= m) {
      tm = first + in % kVocabGroup;
      tn = in / kVocabGroup;
    } else {
      const int rows = m - first;
      tn = in / rows;
      tm = first + in % rows;
    }
  }
};

// The walk of one pair over its units of a launch.  Gradients, launch i: dW
// and dX of piece i - 1, whose G the last launch has just written, then Grad
// of piece i.
template <bool FORWARD>
struct Walk {
  int stage, j, pair, pairs;
  int tiles_m, tiles_n, steps;       // Stats or Grad
  int dw_m, dw_n, dw_steps, splits;  // Dw
  int dx_m, dx_n, dx_steps, line;    // Dx; line: a whole piece's steps
  int whole, x, x1, slot;            // whole: tiles before the line's
  int grad_v0, grad_n, back_v0, back_n;
  int wide, dw_wide;
  bool dx_first;
  Tiles tiles, dw_tiles, dx_tiles;

  __device__ __forceinline__ Walk(const VocabCall& p, int rows, int phase,
                                  int pair_, int pairs_)
      : stage(FORWARD ? 3 : 0), j(pair_), pair(pair_), pairs(pairs_) {
    const VocabHeader* h = p.header;
    grad_v0 = phase * p.piece;
    // (kept logits: G is made outside)
    grad_n = phase < p.pieces && !p.logits ? min(p.piece, p.V - grad_v0) : 0;
    back_v0 = grad_v0 - p.piece;
    back_n = phase > 0 ? min(p.piece, p.V - back_v0) : 0;
    tiles_m = vocab_tiles(rows);
    wide = h ? h->wide : p.wide;
    tiles_n = ((FORWARD ? p.V : grad_n) + wide - 1) / wide;
    steps = vocab_steps(p.D);
    tiles.set(tiles_m, tiles_n);
    dx_first = false;
    if (!FORWARD && phase == 0) {
      stage = 3;
      j = pairs - 1 - pair;
    } else if (!FORWARD) {
      dx_n = vocab_tiles(p.D);
      dw_wide = h->dw_wide;
      dw_n = (p.D + dw_wide - 1) / dw_wide;
      dw_m = vocab_tiles(back_n);
      dw_steps = vocab_steps(rows);
      splits = h->dw_splits;
      dw_tiles.set(dw_m, dw_n);
      dx_m = tiles_m;
      dx_tiles.set(dx_m, dx_n);
      dx_steps = vocab_steps(back_n);
      line = vocab_steps(p.piece);
      whole = h->dx_rounds * pairs;
      x = h->share[pair].x0;
      x1 = h->share[pair].x1;
      slot = h->share[pair].slot;
      dx_first = tiles_m == 1 && (pair & 1);
      if (dx_first) stage = 1;
    }
  }

  // Whether some sum of dW or dX may be deeper than `most` (asked before the
  // first of them).
  __device__ __forceinline__ bool deep(int most) const {
    return (dw_steps + splits - 1) / splits > most ||
           (dx_steps > most && (whole > 0 || x1 - x > most));
  }

  // dX's whole tiles, then its share of the line
  __device__ __forceinline__ bool next_dx(Unit& u) {
    u.kind = kDx;
    u.wide = kVocabTile;
    if (j < whole) {
      dx_tiles.coords(j, u.tm, u.tn);
      u.kb0 = 0;
      u.kb1 = dx_steps;
      u.slot = 0;
      j += pairs;
      return true;
    }
    if (x >= x1) return false;
    const int tile = x / line;
    const int end = min(x1, (tile + 1) * line);
    dx_tiles.coords(whole + tile, u.tm, u.tn);
    // a shorter last piece is cut in proportion
    u.kb0 = x - tile * line;
    u.kb1 = end - tile * line;
    if (dx_steps != line) {
      u.kb0 = (int)((long long)u.kb0 * dx_steps / line);
      u.kb1 = (int)((long long)u.kb1 * dx_steps / line);
    }
    u.slot = slot;
    slot = 0;
    x = end;
    return true;
  }

  __device__ __forceinline__ bool next(Unit& u) {
    if (dx_first && stage == 1) {
      if (next_dx(u)) return true;
      stage = 0;
      j = pair;
    }
    if (stage == 0) {
      const int all = dw_m * dw_n;
      if (j < all * splits) {
        u.kind = kDw;
        u.wide = dw_wide;
        u.slot = 0;
        u.kb0 = 0;
        u.kb1 = dw_steps;
        if (splits > 1) {
          u.slot = j / all;
          // (a depth of below 2^25 steps, 16 splits at most)
          u.kb0 = dw_steps * u.slot / splits;
          u.kb1 = dw_steps * (u.slot + 1) / splits;
        }
        dw_tiles.coords(j - u.slot * all, u.tm, u.tn);
        j += pairs;
        return true;
      }
      stage = dx_first ? 2 : 1;
      j = pair;
    }
    if (stage == 1) {
      if (next_dx(u)) return true;
      stage = 2;
    }
    if (stage == 2) {
      stage = 3;
      // the other way round, so that no pair has the last, partly filled
      // round of both dW and G
      j = pairs - 1 - pair;
    }
    return next_logits(u);
  }

  // The logits' tiles, the last of a launch.
  __device__ __forceinline__ bool next_logits(Unit& u) {
    if (j >= tiles_m * tiles_n) return false;
    u.kind = FORWARD ? kStats : kGrad;
    u.wide = wide;
    tiles.coords(j, u.tm, u.tn);
    u.kb0 = 0;
    u.kb1 = steps;
    u.slot = 0;
    j += pairs;
    return true;
  }
};

// What of a row's targets is read a tile ahead: the target itself, or where
// the teacher's entries for its columns start (a tile's second half may lie
// in a block of columns past the vocabulary, where no entry is).
__device__ __forceinline__ int peek(const VocabCall& p, long long t,
                                    int column) {
  if (p.targets) return (int)p.targets[t];
  if (column >= p.V) return (int)(kVocabNone << 16);
  return (int)p.starts[t * p.blocks + (column >> 7)];
}

// A row's entries from a column on, four of them ahead in registers: the
// next id is at hand when one is passed.
struct Entries {
  const int* ids;
  const float* weights;
  int at, top;
  int id[4];
  float q[4];

  __device__ __forceinline__ void none() {
    at = top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) id[i] = INT_MAX;
  }
  // from a column on; seen: what peek found there
  template <bool WEIGHTS>
  __device__ __forceinline__ void start(const VocabCall& p, long long t,
                                        int column, int seen) {
    if (p.targets) {  // one entry of weight 1
      at = 0;
      top = 1;
      id[0] = seen >= column ? seen : INT_MAX;
      id[1] = id[2] = id[3] = INT_MAX;
      q[0] = 1.f;
      return;
    }
    // (columns are looked at 128 at most at a time, all of one block)
    const uint32_t first = (uint32_t)seen >> 16;
    ids = p.ids + t * p.top;
    weights = p.weights + t * p.top;
    at = seen & 0xffff;
    top = first == kVocabNone ? 0 : p.top;
    id[0] = first == kVocabNone ? INT_MAX : (column & ~127) + (int)first;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool here = at + i < top;
      if (i > 0) id[i] = here ? ids[at + i] : INT_MAX;
      if (WEIGHTS) q[i] = here ? weights[at + i] : 0.f;
    }
    while (id[0] < column) pass<WEIGHTS>();  // (columns inside a block)
  }
  template <bool WEIGHTS>
  __device__ __forceinline__ void pass() {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      id[i] = id[i + 1];
      if (WEIGHTS) q[i] = q[i + 1];
    }
    const bool here = at + 4 < top;
    id[3] = here ? ids[at + 4] : INT_MAX;
    if (WEIGHTS) q[3] = here ? weights[at + 4] : 0.f;
    ++at;
  }
};

// f[i], i < 32 differing by lane: a tree of selections.
__device__ __forceinline__ float pick(const float* f, int i) {
  float a[16], b[8], c[4];
#pragma unroll
  for (int j = 0; j < 16; ++j) a[j] = (i & 16) ? f[j + 16] : f[j];
#pragma unroll
  for (int j = 0; j < 8; ++j) b[j] = (i & 8) ? a[j + 8] : a[j];
#pragma unroll
  for (int j = 0; j < 4; ++j) c[j] = (i & 4) ? b[j + 4] : b[j];
  const float d0 = (i & 2) ? c[2] : c[0], d1 = (i & 2) ? c[3] : c[1];
  return (i & 1) ? d1 : d0;
}


// DEEP: sums of dW or dX may be more than kDeepSteps deep.  FEW: G is in two
// parts (kVocabFewTokens).  SCORE: log probabilities; forward, chunk `phase` of
// the rows; gradients, where the epilogue warps make the next piece's G.
template <int AB_TYPE, bool FORWARD, bool DEEP, bool FEW, bool SCORE>
__global__ void __launch_bounds__(kThreads, 1)
    vocab_gemm_kernel(const __grid_constant__ Maps maps,
                      const __grid_constant__ VocabCall p, const int phase,
                      const __grid_constant__ WaitCfg wc) {
  using Sh = Shape<!FORWARD || SCORE>;
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
    prefetch_tmap(&maps.x);
    prefetch_tmap(&maps.w);
    if (!FORWARD) prefetch_tmap(&maps.g_in);
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

  const VocabHeader* header = p.header;
  const int learnt = header ? header->learnt : p.T;
  const int lo = FEW ? header->lo : 0;
  constexpr bool CHUNK = FORWARD && SCORE;
  const int row0 =
      CHUNK ? (int)min((long long)phase * p.chunk, (long long)learnt) : 0;
  const int all_rows =
      CHUNK ? min(learnt - row0, p.chunk) : vocab_rows(learnt, lo);
  Walk<FORWARD> walk(p, all_rows, phase, pair, pairs);
  Unit u;
  int it = 0, i = 0;  // steps and sums so far
  bool ok = true;
  // G of this piece, and of the one before
  const int g_out = (phase & 1) * p.g_rows, g_in = p.g_rows - g_out;
  if (warp == 0) {
    // ---------------------------------------------------------- producer
    if (lane == 0 && !(wc.debug & kDebugStallProducer)) {
      const void* mx =
          header && header->packed ? &maps.xp : &maps.x;
      while (!*abort && walk.next(u)) {
        const int m0 = u.tm * kVocabTile + (int)rank * kHalf;
        const int n0 = u.tn * u.wide + (int)rank * (u.wide >> 1);
        // Boxes of 64 rows or columns: B, one is enough below 256 columns;
        // A, those with learnt tokens in them (what the others' rows of the
        // stage hold reaches no row that is used; 16 tokens against
        // 100000 × 2048: 98 us with the empty ones, 83 without)
        const bool two = u.wide == kVocabTile;
        const int rows = u.kind == kDw ? kVocabTile
                                       : min(all_rows - u.tm * kVocabTile,
                                             kVocabTile);
        const int boxes0 = min((rows + 63) / 64, 2);
        const int boxes1 = max((rows + 63) / 64 - 2, 0);
        const int boxes = rank == 0 ? boxes0 : boxes1;
        const int bytes =
            (boxes0 + boxes1 + (two ? 4 : 2)) * (kPartBytes / 2);
        // operands K-major: x along the depth; else x along the tile
        const bool mn_a = u.kind == kDw;
        const bool mn_b = u.kind == kDw || u.kind == kDx;
        const void* ma = u.kind == kStats || u.kind == kGrad
                             ? mx
                             : (const void*)&maps.g_in;
        const void* mb = u.kind == kDw ? mx : (const void*)&maps.w;
        // rows of G start at g_in, W's at the piece's first column
        const int am = u.kind == kDx ? g_in + m0 : row0 + m0;
        const int ak = u.kind == kDw ? g_in : 0;
        const int bn = u.kind == kGrad ? walk.grad_v0 + n0 : n0;
        const int bk = u.kind == kDx ? walk.back_v0 : 0;
        for (int kb = u.kb0; kb < u.kb1; ++kb) {
          const int s = it % kStages;
          if (it >= kStages &&
              !bounded_wait(empty(s), ((it / kStages) - 1) & 1, wc.limit,
                            abort, 0)) {
            *abort = 1;
            record_status(wc.status, kStatusTimeoutEmpty);
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(full(s), bytes);
          const uint32_t bar = cluster_map(full(s), 0);
          const uint32_t a = sbase + s * kStageBytes, b = a + kPartBytes;
          const int k = kb * kBK;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h < boxes)
              tma_load2_2d(a + h * (kPartBytes / 2), ma, bar,
                           mn_a ? m0 + 64 * h : k,
                           mn_a ? ak + k : am + 64 * h);
            if (h == 0 || two)
              tma_load2_2d(b + h * (kPartBytes / 2), mb, bar,
                           mn_b ? bn + 64 * h : k,
                           mn_b ? bk + k : bn + 64 * h);
          }
          ++it;
        }
      }
    }
  } else if (warp == 1) {
    // -------------------------------------------------------- MMA issuer
    if (lane == 0 && rank == 0) {
      while (ok && walk.next(u)) {
        const bool mn_a = u.kind == kDw;
        const bool mn_b = u.kind == kDw || u.kind == kDx;
        const uint32_t idesc =
            idesc_f16(256, u.wide, AB_TYPE, mn_b) | (mn_a ? 1u << 15 : 0u);
        // 16 k: 32 bytes along a K-major row, 16 rows of 128 bytes else
        const uint32_t step_a = mn_a ? 2048 : 32, step_b = mn_b ? 2048 : 32;
        int kb = u.kb0;
        const int most = u.kind == kStats || u.kind == kGrad
                             ? sum_steps(p, learnt)
                             : kDeepSteps;
        do {  // one sum; several to a deep tile
          const int end = u.kb1 - kb > most ? kb + most : u.kb1;
          const int b = i & 1;
          if (i >= 2 && !bounded_wait(acc_empty(b), ((i >> 1) - 1) & 1, wc.limit,
                                      abort, 0)) {
            *abort = 1;
            record_status(wc.status, kStatusTimeoutMma);
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t d_tmem = tmem + b * 256;
          for (const int k0 = kb; kb < end; ++kb, ++it) {
            const int s = it % kStages;
            if (!bounded_wait(full(s), (it / kStages) & 1, wc.limit, abort,
                              0)) {
              *abort = 1;
              record_status(wc.status, kStatusTimeoutFull);
              ok = false;
              break;
            }
            tc_fence_after_sync();
            const uint32_t a0 = sbase + s * kStageBytes;
            const uint32_t b0 = a0 + kPartBytes;
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk)
              mma2_f16_ss(d_tmem,
                          smem_desc_sw128(a0 + step_a * kk, kPartBytes / 2,
                                          1024),
                          smem_desc_sw128(b0 + step_b * kk, kPartBytes / 2,
                                          1024),
                          idesc, kb != k0 || kk != 0);
            tc_commit2(empty(s));
          }
          if (ok) tc_commit2(acc_full(b));
          ++i;
        } while (ok && kb < u.kb1);
      }
    }
  } else {
    // ---------------------------------------------------------- epilogue
    const int q = warp & 3;         // TMEM lane quarter
    const int h = (warp - 2) >> 2;  // column half
    const uint32_t my_tmem = tmem + ((uint32_t)(q * 32) << 16);
    const float c2 = p.inv_tau * kLog2e;
    // G of the next piece, of kept logits: runs of columns of it, every
    // warp's in turn, while it has nothing else to do.  (As a kernel of its own
    // it took 61 us beside 132 us of products, 8192 × 32000 × 768.)
    constexpr bool MAKE_G = !FORWARD && SCORE;
    long long run = 0, run_end = 0;
    int runs = 1;
    if (MAKE_G && phase < p.pieces) {
      runs = (min(p.piece, p.V - walk.grad_v0) + kVocabGRun - 1) / kVocabGRun;
      run = (long long)blockIdx.x * kEpiWarps + warp - 2;
      run_end = (long long)((learnt + 63) / 64 * 64) * runs;
    }
    auto make_run = [&]() {
      const int r = (int)(run / runs), at = (int)(run - (long long)r * runs);
      const int cols = min(p.piece, p.V - walk.grad_v0);
      score_g_run<AB_TYPE>(
          p, static_cast<uint16_t*>(p.G) + (long long)g_out * p.piece, r,
          at * kVocabGRun, walk.grad_v0, cols, (cols + 63) / 64 * 64, 0,
          r < learnt, lane, [&](float4& of, int& goal) {
            of = p.terms[r];
            goal = p.goals[r];
          });
      run += (long long)gridDim.x * kEpiWarps;
    };
    // waits for the next sum; its accumulator's address.  (between: of a tile's
    // sums, whose join is in registers)
    auto arrived = [&](uint32_t& acc, auto between) -> bool {
      const int b = i & 1;
      if constexpr (MAKE_G && !decltype(between)::value) {
        while (ok && run < run_end &&
               !__any_sync(0xffffffffu,
                           mbar_test_wait(acc_full(b), (i >> 1) & 1)))
          make_run();
      }
      const bool here = ok && bounded_wait(acc_full(b), (i >> 1) & 1,
                                           wc.limit, abort, kSleepNs);
      if (!__all_sync(0xffffffffu, here)) {
        *abort = 1;
        if (ok && lane == 0) record_status(wc.status, kStatusTimeoutMma);
        ok = false;
        return false;
      }
      tc_fence_after_sync();
      acc = my_tmem + b * 256;
      return true;
    };
    // this warp's part of the accumulator is in registers
    auto release = [&]() {
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_pair(cluster_map(acc_empty(i & 1), 0));
      ++i;
    };

    // Several sums of a tile: added here, and put in the last one's place.
    // (acc: its address, this warp's columns; idle: nobody reads them.)
    auto join_sums = [&](int half, int steps, int most, uint32_t& acc,
                         bool idle = false) -> bool {
      if (!arrived(acc, std::false_type())) return false;
      acc += h * half;
      float f[128];
#pragma unroll
      for (int c = 0; c < 128; ++c) f[c] = 0.f;
      for (;; steps -= most) {
#pragma unroll
        for (int c = 0; c < 128; c += 16) {
          if (c >= half || idle) break;
          uint32_t v[16];
          if (tmem_span_ok(acc + c, 16, tmem, kTmemCols, q, wc.status))
            tmem_ld16(acc + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) f[c + j] += __uint_as_float(v[j]);
        }
        if (steps <= most) break;
        release();
        if (!arrived(acc, std::true_type())) return false;
        acc += h * half;
      }
#pragma unroll
      for (int c = 0; c < 128; c += 16) {
        if (c >= half || idle) break;
        tmem_st16(acc + c, reinterpret_cast<const uint32_t*>(f + c));
      }
      tmem_st_wait();
      return true;
    };

    // The first pass is a dry run, on whatever TMEM holds and
    // with nothing stored: it brings the instructions in while the first
    // tile is being made (which they otherwise hold up by 2-3 us).
    bool first_pass = true;
    // The next tile, and of this row's targets in it what costs a load to
    // find: read while the tile before is worked on.
    Unit nu;
    int n_token = 0, n_seen = 0;
    float n_lse = 0.f, n_grad = 0.f;
    auto look_ahead = [&](auto in_logits) -> bool {
      if (!(decltype(in_logits)::value ? walk.next_logits(nu) : walk.next(nu)))
        return false;
      int r = row0 + nu.tm * kVocabTile + (int)rank * kHalf + q * 32 + lane;
      if (FEW && r >= lo) r -= lo;  // (both parts are one token's)
      if ((nu.kind == kStats || nu.kind == kGrad) && r < learnt) {
        n_token = learnt == p.T ? r : p.token[r];
        const int n0 = nu.tn * nu.wide + h * (nu.wide >> 1);
        n_seen = peek(p, n_token, FORWARD ? n0 : walk.grad_v0 + n0);
        if (!FORWARD) {
          n_lse = p.lse[n_token];
          n_grad = p.grad_loss[n_token * p.grad_stride];
        }
      }
      return true;
    };
    // staging: row (lane) of 128 bytes, its 16-byte chunk j at j ^ (row
    // mod 8), the layout a 128-byte-swizzle TMA store reads
    unsigned char* stg = smem + Sh::kOffStaging + (warp - 2) * kStagingBytes;
    const uint32_t stg_s =
        sbase + Sh::kOffStaging + (warp - 2) * kStagingBytes;
    // 32 columns of fp32: one staged block
    auto stage_32 = [&](const float* f) {
      if (lane == 0) bulk_wait_group_read<0>();
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<float4*>(stg + lane * 128 + ((j ^ (lane & 7)) << 4)) =
            make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
      fence_proxy_async_smem();
      __syncwarp();
    };
    const bool deep = DEEP && phase > 0 && walk.deep(kDeepSteps);
    bool more = look_ahead(std::false_type());
    if constexpr (FORWARD) {
      const int most = sum_steps(p, learnt);
      for (;; first_pass = false) {
        int token = 0, seen = 0;
        if (first_pass) {
          u = {kStats, 1 << 20, 0, 64, 0, 0, 0};
        } else {
          if (!more) break;
          u = nu;
          token = n_token;
          seen = n_seen;
        }
        const int m0 = u.tm * kVocabTile + (int)rank * kHalf + q * 32;
        const int r = row0 + m0 + lane;
        const int half = u.wide >> 1;  // this warp's columns
        const int n0 = u.tn * u.wide + h * half;
        uint32_t acc = my_tmem;
        const bool several = u.kb1 > most;
        // No row of this warp's is a token's: it has nothing to do but to let
        // the accumulators go (one token 128000 × 4096: 196 us without this,
        // 189 with).
        const bool idle = SCORE && !first_pass && m0 >= all_rows;
        if (several && !join_sums(half, u.kb1, most, acc, idle)) break;
        if (!first_pass) more = look_ahead(std::true_type());
        Entries e;
        e.none();
        if (!first_pass && r < learnt) e.start<false>(p, token, n0, seen);
        // the warp's first entry: most stretches of columns have none
        int next = __reduce_min_sync(0xffffffffu, e.id[0]);
        if (!several) {
          if (!first_pass && !arrived(acc, std::false_type())) break;
          acc += h * half;
        }
        if (idle) {
          release();
          continue;
        }
        float peak = -INFINITY, sum = 0.f;
        float slant = 0.f, largest = -INFINITY;  // (SCORE)
#pragma unroll 1
        for (int c = 0; c < half; c += 32) {
          const int n = n0 + c;
          float f[32];
          {
            uint32_t v[32];
            if (tmem_span_ok(acc + c, 32, tmem, kTmemCols, q, wc.status))
              tmem_ld32(acc + c, v);
            tmem_ld_wait();
            if (c + 32 == half && !first_pass) release();
#pragma unroll
            for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[j]);
          }
          if (n >= p.V) continue;  // (after the release)
          while (next < n + 32) {
            if (e.id[0] < n + 32) {
              float* to = p.picked + (long long)r * p.top + e.at;
              if (span_ok(to, 4, p.picked, 4ll * p.T * p.top, wc.status))
                *to = pick(f, e.id[0] - n) * (SCORE ? 1.f : p.inv_tau);
              e.pass<false>();
            }
            next = __reduce_min_sync(0xffffffffu, e.id[0]);
          }
          if (SCORE && p.logits) {
            stage_32(f);
            if (lane == 0) {
              if (!first_pass && m0 < all_rows)
                tma_store_2d(&maps.logits, stg_s, n, m0);
              bulk_commit_group();
            }
          }
          if (n + 32 > p.V) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (n + j >= p.V) f[j] = -INFINITY;
          }
          float top4[4] = {f[0], f[1], f[2], f[3]};
#pragma unroll
          for (int j = 4; j < 32; ++j) top4[j & 3] = fmaxf(top4[j & 3], f[j]);
          const float here =
              fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
          const float now = fmaxf(peak, here * c2);
          // a stretch of -Inf only: every term is 0, not exp(-Inf + Inf)
          const float ref = now == -INFINITY ? 0.f : now;
          scale_add_32(f, c2, -ref);
          if constexpr (SCORE) {
            // Σ e·log2 e, e = 2^(z·c2 - ref): from the last reference to this
            // one a term's logarithm moves by d.
            const float d = fmaxf(peak - ref, -1e30f), keep = exp2_fast(d);
            float e[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) e[j] = exp2_fast(f[j]);
            float more = dot_32(e, f);
            if (more != more) {
              // A logit of -Inf has e = 0, and here no logarithm below -1e30:
              // their product is 0.  (A NaN stays in e.  The limit on every
              // logit took 2 % more time: 8192 × 32000 × 768 292 us.)
#pragma unroll
              for (int j = 0; j < 32; ++j) f[j] = fmaxf(f[j], -1e30f);
              more = dot_32(e, f);
            }
            slant = keep * (slant + d * sum) + more;
            sum = sum * keep + sum_32(e);
            largest = fmaxf(largest, here);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) f[j] = exp2_fast(f[j]);
            sum = sum * exp2_fast(peak - ref) + sum_32(f);
          }
          peak = now;
        }
        if (first_pass || n0 >= p.V) continue;
        const int parts = (int)((2ll * p.V + u.wide - 1) / u.wide);
        if constexpr (SCORE) {
          // (a row's are read together)
          float4* to = p.sums + (long long)r * parts + u.tn * 2 + h;
          if (r < learnt &&
              span_ok(to, 16, p.sums, 16ll * parts * learnt, wc.status))
            *to = make_float4(peak, sum, slant, largest);
        } else {
          float2* to = p.stats + (long long)(u.tn * 2 + h) * learnt + r;
          if (r < learnt &&
              span_ok(to, 8, p.stats, 8ll * parts * learnt, wc.status))
            *to = make_float2(peak, sum);
        }
      }
      if (SCORE && lane == 0) bulk_wait_group<0>();
    } else {
      const float inv_scale = header->inv_scale;
      const float grad_scale = p.tau * header->scale;
      const bool dw_direct = !p.dWp && !vocab_maps(p.dW, p.lddw);
      const int slot_rows = vocab_tiles(learnt) * kVocabTile;
      const int most = sum_steps(p, learnt);
      // dW's and dX's tiles, then the logits': a loop each, so that the sums
      // of the logits share their registers with little else; and one for
      // tiles of dW and dX that are several sums, which holds too much beside
      // these not to spill.  (It is in a kernel of its own: 8192 × 1000 × 512
      // distillation steps took 4 us more with it in the code.)
      auto epilogues = [&](auto loop) {
        constexpr bool LOGITS = decltype(loop)::value == kLogits;
        constexpr bool DEEP_LOOP = decltype(loop)::value == kDeep;
        for (;; first_pass = false) {
          int token = 0, seen = 0;
          float shift = 0.f, g = 0.f;
          if (first_pass) {
            u = {LOGITS ? kGrad : kDx, 1 << 20, 0, 128, 0, 1, 0};
          } else {
            if (!more || (nu.kind == kGrad) != LOGITS) break;
            u = nu;
            token = n_token;
            seen = n_seen;
            // g·p is one exponential, 2^(z·c2 + log2 |g| - lse·log2 e), with
            // g's sign (g = 0: the exponent is -Inf)
            g = n_grad * grad_scale;
            shift = log2f(fabsf(g)) - n_lse * kLog2e;
          }
          uint32_t acc = my_tmem;
          const int wide_here = LOGITS && !first_pass ? walk.wide : u.wide;
          const int half = wide_here >> 1;  // this warp's columns
          const int steps = LOGITS ? walk.steps : u.kb1 - u.kb0;
          const bool several = (LOGITS || DEEP_LOOP) && !first_pass &&
                               steps > (LOGITS ? most : kDeepSteps);
          if (several &&
              !join_sums(half, steps, LOGITS ? most : kDeepSteps, acc))
            break;
          if (!first_pass) more = look_ahead(std::bool_constant<LOGITS>());
          const int m0 = u.tm * kVocabTile + (int)rank * kHalf + q * 32;
          // this warp's rows are the second parts of G's
          const bool second = FEW && LOGITS && m0 >= lo;
          const int r = m0 + lane - (second ? lo : 0);
          const int n0 = u.tn * wide_here + h * half;
          // G is written to the end of its tiles
          const int cols = LOGITS ? INT_MAX : p.D;
          Entries e;
          e.none();
          if (LOGITS && !first_pass && r < learnt)
            e.start<true>(p, token, walk.grad_v0 + n0, seen);
          int next = __reduce_min_sync(0xffffffffu, e.id[0]);
          // sums in fp32 slots
          const bool wide =
              !LOGITS && (u.kind == kDx || header->dw_splits > 1);
          if (!several) {
            if (!first_pass && !arrived(acc, std::false_type())) break;
            acc += h * half;
          }
          if (!LOGITS && u.kind == kDw && !wide && !dw_direct) {
            // Nothing to work out: 64 columns at a time, packed and stored.
            // With few tokens a tile is its epilogue alone, which waits for
            // itself more than for anything else (16 tokens, 100000 × 2048: a
            // step took 22 us more, of 330, with 32 columns at a time as
            // below).
#pragma unroll 1
            for (int c0 = 0; c0 < half; c0 += 64) {
              uint32_t v[64];
              if (tmem_span_ok(acc + c0, 64, tmem, kTmemCols, q,
                               wc.status)) {
                tmem_ld32(acc + c0, v);
                tmem_ld32(acc + c0 + 32, v + 32);
              }
              tmem_ld_wait();
              if (c0 + 64 == half) release();
              const int n = n0 + c0;
              if (n >= p.D) continue;  // (after the release)
              if (lane == 0) bulk_wait_group_read<0>();
              __syncwarp();
              const bool empty = u.kb0 == u.kb1;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float lo = __uint_as_float(v[8 * j + 2 * k]);
                  const float hi = __uint_as_float(v[8 * j + 2 * k + 1]);
                  w[k] =
                      empty ? 0u : pack16_scaled<AB_TYPE>(lo, hi, inv_scale);
                }
                *reinterpret_cast<uint4*>(stg + lane * 128 +
                                          ((j ^ (lane & 7)) << 4)) =
                    make_uint4(w[0], w[1], w[2], w[3]);
              }
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                if (m0 < walk.back_n)
                  tma_store_2d(&maps.dw, stg_s, n, walk.back_v0 + m0);
                bulk_commit_group();
              }
            }
            continue;
          }
#pragma unroll 1
          for (int c0 = 0; c0 < half; c0 += 32) {
            uint32_t v[32];
            if (tmem_span_ok(acc + c0, 32, tmem, kTmemCols, q,
                             wc.status))
              tmem_ld32(acc + c0, v);
            tmem_ld_wait();
            if (c0 + 32 == half && !first_pass) release();
            const int n = n0 + c0;
            if (n >= cols) continue;  // (after the release)
            float f[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[j]);
            if (LOGITS) {
              scale_add_32(f, c2, shift);
#pragma unroll
              for (int j = 0; j < 32; ++j) f[j] = exp2_fast(f[j]);
              // columns past the vocabulary are zeros, and (below) rows past
              // the learnt tokens: Dw and Dx sum over them up to multiples of
              // 64
              if (n + 32 > walk.grad_n) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (n + j >= walk.grad_n) f[j] = 0.f;
              }
            } else if (u.kb0 == u.kb1) {  // an empty sum
#pragma unroll
              for (int j = 0; j < 32; ++j) f[j] = 0.f;
            }
            if (wide) {
              stage_32(f);
              if (lane == 0) {
                if (u.kind == kDx) {
                  if (!first_pass && m0 < all_rows) {
                    if (phase == 1)  // the first piece
                      tma_store_2d(&maps.slots, stg_s, n,
                                   u.slot * slot_rows + m0);
                    else
                      tma_add_2d(&maps.slots, stg_s, n,
                                 u.slot * slot_rows + m0);
                  }
                } else if (m0 < walk.back_n) {
                  tma_store_2d(&maps.dw_slots, stg_s, n,
                               u.slot * p.dw_slot_rows + m0);
                }
                bulk_commit_group();
              }
              continue;
            }
            // 16-bit, 64 columns: half a staged block at a time
            if (!LOGITS) {
#pragma unroll
              for (int j = 0; j < 32; ++j) f[j] *= inv_scale;
            }
            if ((c0 & 32) == 0) {
              if (lane == 0) bulk_wait_group_read<0>();
              __syncwarp();
            }
            uint32_t keep = 0xffffffffu, flip = 0;
            if (LOGITS) {
              keep = r < learnt ? 0xffffffffu : 0u;
              flip = g < 0.f ? 0x80008000u : 0u;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int chunk = (c0 & 32) / 8 + j;
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float a = f[8 * j + 2 * k], b = f[8 * j + 2 * k + 1];
                w[k] = pack16<AB_TYPE>(a, b);
                if (second) w[k] = pack16_rest<AB_TYPE>(a, b, w[k]);
                w[k] = (w[k] ^ flip) & keep;
              }
              *reinterpret_cast<uint4*>(stg + lane * 128 +
                                        ((chunk ^ (lane & 7)) << 4)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
            if (LOGITS) {
              // the row's targets in these columns: p - q, in their places
              const int column = walk.grad_v0 + n;
              float part = 0.f;
              while (next < column + 32) {
                if (e.id[0] < column + 32) {
                  const int c = e.id[0] - column;
                  part += e.q[0];  // an id may come again
                  e.pass<true>();
                  if (e.id[0] != column + c) {
                    const int chunk = (c0 & 32) / 8 + (c >> 3);
                    unsigned char* to = stg + lane * 128 +
                                        ((chunk ^ (lane & 7)) << 4) +
                                        (c & 7) * 2;
                    if (span_ok(to, 2, stg, kStagingBytes, wc.status)) {
                      const float v = copysignf(pick(f, c), g) - g * part;
                      uint32_t w = pack16<AB_TYPE>(v, 0.f);
                      if (second) w = pack16_rest<AB_TYPE>(v, 0.f, w);
                      *reinterpret_cast<uint16_t*>(to) = (uint16_t)w;
                    }
                    part = 0.f;
                  }
                }
                next = __reduce_min_sync(0xffffffffu, e.id[0]);
              }
            }
            // the block is whole, or its other half lies past the columns
            if ((c0 & 32) == 0 && n + 32 < cols) continue;
            const int nb = n - (c0 & 32);
            if (!LOGITS && dw_direct) {
              // rows on any 2-byte boundary, and no room for them elsewhere: a
              // warp writes 64 columns of one row at a time
              __syncwarp();
              const int rows = min(32, walk.back_n - m0);
              for (int k = 0; k < rows; ++k) {
                const uint32_t two = *reinterpret_cast<const uint32_t*>(
                    stg + k * 128 + (((lane >> 2) ^ (k & 7)) << 4) +
                    (lane & 3) * 4);
                uint16_t* to =
                    static_cast<uint16_t*>(p.dW) +
                    (long long)(walk.back_v0 + m0 + k) * p.lddw + nb +
                    2 * lane;
                if (nb + 2 * lane >= cols ||
                    !span_ok(to, min(4, 2 * (cols - nb - 2 * lane)), p.dW,
                             2 * ((p.V - 1) * p.lddw + p.D), wc.status))
                  continue;
                if (nb + 2 * lane + 1 < cols &&
                    (reinterpret_cast<uintptr_t>(to) & 3u) == 0) {
                  *reinterpret_cast<uint32_t*>(to) = two;
                } else {
                  to[0] = (uint16_t)two;
                  if (nb + 2 * lane + 1 < cols) to[1] = (uint16_t)(two >> 16);
                }
              }
              __syncwarp();
            } else {
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                if (LOGITS) {
                  if (!first_pass)
                    tma_store_2d(&maps.g_out, stg_s, nb, g_out + m0);
                } else if (m0 < walk.back_n)
                  tma_store_2d(&maps.dw, stg_s, nb, walk.back_v0 + m0);
                bulk_commit_group();
              }
            }
          }
        }
      };
      if (phase > 0) {
        if (deep) {
          if constexpr (DEEP) epilogues(std::integral_constant<Loop, kDeep>());
        } else {
          epilogues(std::integral_constant<Loop, kShallow>());
        }
      }
      if constexpr (MAKE_G) {
        while (ok && run < run_end) make_run();
      } else if (phase < p.pieces && !p.logits) {
        epilogues(std::integral_constant<Loop, kLogits>());
      }
      if (lane == 0) bulk_wait_group<0>();
    }
  }

  if (lane == 0 && rank == 0 && warp == 0 && *abort) {
    // let the copies still in flight land
    for (int k = it > kStages ? it - kStages : 0; k < it; ++k)
      if (!bounded_wait(full(k % kStages), (k / kStages) & 1, kDrainNs,
                        nullptr, 0))
        record_status(wc.status, kStatusTimeoutDrain);
  }
  // the last arrival in both CTAs
  if (lane == 0 && rank == 0 && warp == 1) tc_commit2(mma_done);
  griddep_launch_dependents();
  tc_fence_before_sync();
  __syncwarp();  // reconverge the warps whose roles ran on one lane
  __syncthreads();
  // No product may still run when TMEM is freed, nor signal a CTA that has
  // left.  Waited for here, when this CTA's epilogues are over and the last
  // products with them: the second CTA's warp 1 has no other role, and a limit
  // that began with the kernel would bound the whole launch.
  if (warp == 1 && lane == 0 &&
      !bounded_wait(mma_done, 0, kDrainNs, nullptr, 0))
    record_status(wc.status, kStatusTimeoutDrain);
  __syncwarp();
  cluster_sync_all();  // the pair's products and copies are over
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc2(tmem, kTmemCols);
  }
}

// A row-major matrix (x contiguous), 128-byte-wide boxes of `by` rows in the
// 128-byte swizzle; elements outside read as zeros and are not written.
bool encode(CUtensorMap* m, CUtensorMapDataType type, int size,
            const void* base, long long x, long long y, long long ld, int by) {
  const cuuint64_t dims[2] = {(cuuint64_t)x, (cuuint64_t)y};
  const cuuint64_t strides[1] = {(cuuint64_t)(ld * size)};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / size), (cuuint32_t)by};
  const cuuint32_t estr[2] = {1, 1};
  return tensor_map_encoder()(
             m, type, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int AB_TYPE>
bool make_maps(const VocabCall& p, bool grad, Maps* maps) {
  const CUtensorMapDataType t16 = AB_TYPE == 1
                                      ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const CUtensorMapDataType t32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  if (!tensor_map_encoder()) return false;
  std::memset(maps, 0, sizeof(*maps));
  bool ok = p.Wp ? encode(&maps->w, t16, 2, p.Wp, p.D, p.V, p.ldxp, 64)
                 : encode(&maps->w, t16, 2, p.W, p.D, p.V, p.ldw, 64);
  if (p.header)
    ok = ok && encode(&maps->xp, t16, 2, p.Xp, p.D, p.xp_rows, p.ldxp, 64);
  // X as given may have no tensor map: then only the packed copy is read
  if (vocab_maps(p.X, p.ldx))
    ok = ok && encode(&maps->x, t16, 2, p.X, p.D, p.T, p.ldx, 64);
  if (!grad && p.logits)
    ok = ok && encode(&maps->logits, t32, 4, p.logits, p.V, p.chunk,
                      p.ld_logits, 32);
  if (!grad) return ok;
  const long long g_rows = (p.pieces > 1 ? 2ll : 1ll) * p.g_rows;
  ok = ok && encode(&maps->g_in, t16, 2, p.G, p.piece, g_rows, p.piece, 64) &&
       encode(&maps->g_out, t16, 2, p.G, p.piece, g_rows, p.piece, 32) &&
       encode(&maps->slots, t32, 4, p.slots, p.D, p.slot_rows, p.ld_slot, 32);
  if (p.dw_slots)
    ok = ok && encode(&maps->dw_slots, t32, 4, p.dw_slots, p.D,
                      (long long)p.dw_slot_rows * p.dw_max_splits, p.ld_slot,
                      32);
  if (p.dWp)
    ok = ok && encode(&maps->dw, t16, 2, p.dWp, p.D, p.V, p.ldxp, 32);
  else if (vocab_maps(p.dW, p.lddw))
    ok = ok && encode(&maps->dw, t16, 2, p.dW, p.D, p.V, p.lddw, 32);
  return ok;
}

// Launches first to last - 1.
template <int AB_TYPE, bool FORWARD, bool DEEP = false, bool FEW = false,
          bool SCORE = false>
cudaError_t launch(const VocabCall& p, const WaitCfg& wc, cudaStream_t stream,
                   int first = 0, int last = 1) {
  using Sh = Shape<!FORWARD || SCORE>;
  Maps maps;
  if (!make_maps<AB_TYPE>(p, !FORWARD, &maps)) return cudaErrorInvalidValue;
  auto fn = vocab_gemm_kernel<AB_TYPE, FORWARD, DEEP, FEW, SCORE>;
  cudaError_t e =
      ensure_smem_attr(reinterpret_cast<const void*>(fn), Sh::kSmemBytes);
  for (int phase = first; phase < last && e == cudaSuccess; ++phase) {
    // the piece's G, but where the launch before made it
    if (!FORWARD && p.logits && (!SCORE || phase == first))
      e = vocab_score_g(p, phase - 1, 2 * p.pairs, stream);
    if (e == cudaSuccess)
      e = launch_pdl_cluster(fn, dim3(2 * p.pairs), dim3(kThreads),
                             Sh::kSmemBytes, stream, 2, maps, p, phase, wc);
  }
  return e;
}

}  // namespace vocab

cudaError_t vocab_forward(const VocabCall& c, const WaitCfg& wc,
                          cudaStream_t stream) {
  return c.type == GEMM_F32_MIXED_BF16 ? vocab::launch<1, true>(c, wc, stream)
                                       : vocab::launch<0, true>(c, wc, stream);
}

cudaError_t vocab_score(const VocabCall& c, const WaitCfg& wc, int phase,
                        cudaStream_t stream) {
  using vocab::launch;
  return c.type == GEMM_F32_MIXED_BF16
             ? launch<1, true, false, false, true>(c, wc, stream, phase,
                                                   phase + 1)
             : launch<0, true, false, false, true>(c, wc, stream, phase,
                                                   phase + 1);
}

cudaError_t vocab_gradients(const VocabCall& c, const WaitCfg& wc,
                            cudaStream_t stream) {
  // dW sums over the tokens, dX over a piece's words
  const bool deep =
      std::max(vocab_steps(c.T), vocab_steps(c.piece)) > vocab::kDeepSteps;
  const bool few = c.T <= kVocabFewTokens;
  // (of kept logits, no launch makes G alone)
  const int first = c.logits ? 1 : 0, last = c.pieces + 1;
  using vocab::launch;
  if (c.logits && !few) {
    if (c.type == GEMM_F32_MIXED_BF16)
      return deep ? launch<1, false, true, false, true>(c, wc, stream, first,
                                                        last)
                  : launch<1, false, false, false, true>(c, wc, stream, first,
                                                         last);
    return deep ? launch<0, false, true, false, true>(c, wc, stream, first,
                                                      last)
                : launch<0, false, false, false, true>(c, wc, stream, first,
                                                       last);
  }
  if (c.type == GEMM_F32_MIXED_BF16)
    return few    ? launch<1, false, true, true>(c, wc, stream, first, last)
           : deep ? launch<1, false, true>(c, wc, stream, first, last)
                  : launch<1, false>(c, wc, stream, first, last);
  return few    ? launch<0, false, true, true>(c, wc, stream, first, last)
         : deep ? launch<0, false, true>(c, wc, stream, first, last)
                : launch<0, false>(c, wc, stream, first, last);
}

}  // namespace gemm_f32_impl
