// Log probabilities of given words, entropy and the likeliest words: what
// surrounds their products (vocab_gemm.cu).
//
// With z = X·Wᵀ, c = log2 e / τ and, per row, e_v = 2^(c·z_v − r), r = max c·z,
//   S = Σ e_v,  E = Σ e_v·log2 e_v:
//   lse = ln 2·(r + log2 S),   logp = ln 2·(c·z_y − r − log2 S),
//   entropy = −Σ p·log p = ln 2·(log2 S − E/S).
// The products leave S, E, r and the largest z of each half tile.  (As z_y/τ −
// lse, logp would have lse's rounding, 1e-6 of a probability near 1 whose
// logarithm is 1e-2.)
//
// The likeliest words.  The k largest elements of a row lie in the k stretches
// (half tiles) with the largest maxima, of equal ones the first: any element
// elsewhere has k larger ones before it, or equal ones with lower ids.  So the
// logits are stored, of some tokens at a time, and of each row only those
// stretches are read, about k·128 of V logits.  (Storing them costs the
// products 5 % at width 4096 and 28 % at width 768, 4096 and 8192 tokens; for
// few tokens 2·T/D of the weights' bytes.)
//   The rank of two logits should not hang on how a sum rounds (on the tile it
// was made in, so on the batch): the k + kSpare largest are computed again
// from the operands, products exact in fp32, summed in pairs of fp32 (48
// bits as a rule; ExactSum has the bound), and ranked by that.  A word that is not among them can only belong to
// the first k if its fp32 logit lies within its own error of the k-th exact
// one; where there may be such words (a row in some million: 8 ranks lie far
// further apart) all of them are computed again.
//
// Gradients.  G = (a·([v = y] − p) − b·p·(log p + H))/τ from the kept logits,
// 4 bytes read and 2 written an element, a piece of the vocabulary at a time,
// which then is in L2 for the products: the first piece by a kernel of its own,
// bound by memory, the later ones by the products' epilogue warps, which
// otherwise wait for the tensor cores most of the time (vocab_gemm.cu).  Making
// the logits again would cost 2·D operations an element instead.
//   G is rounded to the operands' 16 bits, which kind::f16 asks for: beyond 128
// tokens once, so that dX and dW are 2.4e-3 off float64 in bfloat16 and 2.9e-4
// in binary16, where rounding the results alone leaves 1.65e-3 and 2.1e-4.  G in
// two parts (vocab.cuh, kVocabFewTokens) would leave that too, for twice the
// operations of both products, two thirds of a step's.
#include <algorithm>

#include "bound_search.h"
#include "gemm_f32.h"
#include "kernels.h"
#include "vocab.cuh"

namespace gemm_f32_impl {
namespace {

constexpr float kLn2 = 0.69314718056f, kLog2e = 1.4426950408889634f;

// Numbers in the order of the floats, from kLowest on; a NaN counts as -Inf.
constexpr uint32_t kLowest = 0x007fffffu;
__device__ __forceinline__ uint32_t order_of(float f) {
  if (f != f) return kLowest;
  const uint32_t u = __float_as_uint(f + 0.f);  // (-0 as 0)
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// ------------------------------------------------------------- statistics
struct Stat {
  float m, s, e;  // r, S, E
};

// What a statistic with the reference m counts for beside one of reference
// `ref`: its logarithms move by d.  (Of nothing: d finite, 0 · d = 0.)
__device__ __forceinline__ float moved(float m, float ref) {
  return fmaxf(m - ref, -1e30f);
}

// The number of an order.
__device__ __forceinline__ float reference_of(uint32_t order) {
  const uint32_t u = order & 0x80000000u ? order ^ 0x80000000u : ~order;
  return __uint_as_float(u);
}

// The statistics of all lanes joined.
__device__ __forceinline__ Stat merge_warp(Stat st) {
  const float m = reference_of(
      __reduce_max_sync(0xffffffffu, order_of(st.m)));
  const float ref = m == -INFINITY ? 0.f : m;
  const float d = moved(st.m, ref), keep = exp2f(d);
  float e = keep * (st.e + d * st.s), s = keep * st.s;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    e += __shfl_xor_sync(0xffffffffu, e, o);
  }
  return Stat{m, s, e};
}

// The statistics first, first + step, ... of row r, with what each addition
// rounds off kept (a large vocabulary is many additions); each one's largest
// logit goes to `largest`.
template <typename Largest>
__device__ __forceinline__ Stat share_of(const VocabCall& p, int r, int first,
                                         int parts, int step,
                                         Largest largest) {
  const float4* sums = p.sums + (long long)r * parts;
  Stat st = {-INFINITY, 0.f, 0.f};
  float lost = 0.f, lost_e = 0.f;
#pragma unroll 4
  for (int g = first; g < parts; g += step) {
    float4 b = make_float4(-INFINITY, 0.f, 0.f, -INFINITY);
    if (span_ok(sums + g, 16, p.sums, 16ll * p.T * parts, p.status))
      b = sums[g];
    largest(g, b.w);
    const float m = fmaxf(st.m, b.x);
    const float ref = m == -INFINITY ? 0.f : m;
    const float da = moved(st.m, ref), db = moved(b.x, ref);
    const float ka = exp2f(da), kb = exp2f(db);
    const float was = st.s * ka, was_e = ka * (st.e + da * st.s);
    const float more = b.y * kb - lost * ka;
    const float more_e = kb * (b.z + db * b.y) - lost_e * ka;
    st = Stat{m, was + more, was_e + more_e};
    lost = (st.s - was) - more;
    lost_e = (st.e - was_e) - more_e;
  }
  return st;
}

// A row's results; z: its word's logit.  What the gradients need of it goes
// behind its kept logits.
__device__ __forceinline__ void store_results(const VocabCall& p, long long t,
                                              int r, bool scored, Stat st,
                                              float log_sum, float z) {
  if (p.keep) {
    float* of_row = p.logits + (long long)r * p.ld_logits + p.V;
    of_row[0] = st.m;
    of_row[1] = log_sum;
  }
  // (the difference of equal numbers where one word has all: not below 0)
  const float entropy = log_sum - kLn2 * (st.e / st.s);
  p.loss[t] = scored ? vocab_log_prob(p, z, st.m, log_sum) : 0.f;
  p.lse_out[t] = scored ? fmaf(kLn2, st.m, log_sum) : 0.f;
  p.entropy_out[t] = scored && !(entropy < 0.f) ? entropy : 0.f;
}

// logp, lse and entropy of the rows from row0 on, a block each.
constexpr int kFinishThreads = 256;
__global__ void __launch_bounds__(kFinishThreads)
    finish_score_kernel(const __grid_constant__ VocabCall p, int row0) {
  __shared__ Stat s_part[kFinishThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int learnt = p.header ? p.header->learnt : p.T;
  const int wide = p.header ? p.header->wide : p.wide;
  const int parts = (int)((2ll * p.V + wide - 1) / wide);  // half tiles
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = row0 + blockIdx.x;
  if (r >= learnt) return;
  const long long t = learnt != p.T ? p.token[r] : r;
  const bool scored = p.header || vocab_is_learnt(p, t);
  const float z = scored ? p.picked[r] : 0.f;
  Stat st = merge_warp(share_of(p, r, threadIdx.x, parts, kFinishThreads,
                                [](int, float) {}));
  if (lane == 0) s_part[warp] = st;
  __syncthreads();
  if (warp > 0) return;
  st = lane < kFinishThreads / 32 ? s_part[lane] : Stat{-INFINITY, 0.f, 0.f};
  st = merge_warp(st);
  if (lane == 0) store_results(p, t, r, scored, st, logf(st.s), z);
}

// ------------------------------------------------------- likeliest words
constexpr int kSpare = 8;  // ranked beyond those asked for
constexpr int kMostRanked = kVocabMaxTop + kSpare;
// What an fp32 logit may be off by, times the sum of its terms' magnitudes: 32
// additions (kind::f16 takes 16 products each, 8 steps of 64 are a sum) short
// of four last places, 2^-21, each, and half a last place, 2^-24, for each sum
// of 512 that is added.  Doubled, as the sum is that of some of the largest
// words, not of all.
__device__ __forceinline__ float logit_error(int D) {
  return 0x1p-15f + 0x1p-32f * (float)D;
}
constexpr int kStretches = 512;    // read at most, but for equal maxima
constexpr int kCandidates = 1024;  // ranked at most, but for equal logits
constexpr int kHeldKeys = 2048;

struct SelectState {
  int hist[256];
  int digit, left;
  int gt[32], eq[32];
};

// The k-th largest of n >= k keys, and how many of those equal to it are among
// the k: 8 bits at a time, from a histogram of the keys that begin as it does.
template <int THREADS, typename Key>
__device__ __forceinline__ uint32_t kth_largest(SelectState& s, int n, int k,
                                                Key key, int& equal) {
  const int tid = threadIdx.x;
  uint32_t prefix = 0;
  int left = k;
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int b = tid; b < 256; b += THREADS) s.hist[b] = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < n; i += THREADS) {
      const uint32_t x = key(i);
      if (shift == 24 || (x ^ prefix) >> (shift + 8) == 0)
        atomicAdd(&s.hist[(x >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid < 32) {  // 8 bins a lane, the largest first
      const int top = 255 - 8 * tid;
      int sum = 0;
#pragma unroll
      for (int b = 0; b < 8; ++b) sum += s.hist[top - b];
      int upto = sum;
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (tid >= o) upto += v;
      }
      int before = upto - sum;
      if (before < left && left <= upto) {
        int b = 0;
        while (before + s.hist[top - b] < left) before += s.hist[top - b++];
        s.digit = top - b;
        s.left = left - before;
      }
    }
    __syncthreads();
    prefix |= (uint32_t)s.digit << shift;
    left = s.left;
    __syncthreads();
  }
  equal = left;
  return prefix;
}

// A bound that at least k of n >= k keys from low on reach, and not many more
// (bound_search.h).  (Keys of one row mostly differ in their last 24 bits: a
// histogram of the first 8 would have one bin, and every atomic on it in turn.)
template <int THREADS, typename Key>
__device__ __forceinline__ uint32_t reached_by(SelectState& s, int n, int k,
                                               uint32_t low, uint32_t high,
                                               Key key) {
  constexpr int kEnough = 32;
  const int tid = threadIdx.x;
  auto count = [&](uint32_t low, uint32_t high, int shift, int& in_step) {
    for (int b = tid; b < kBoundBins; b += THREADS) s.hist[b] = 0;
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < n; i += THREADS) {
      const uint32_t x = key(i);
      if (x >= low) atomicAdd(&s.hist[bound_bin(x, low, high, shift)], 1);
    }
    __syncthreads();
    if (tid < 32) {  // 8 bins a lane, the largest first
      const int top = 255 - 8 * tid;
      int sum = 0;
#pragma unroll
      for (int b = 0; b < 8; ++b) sum += s.hist[top - b];
      int upto = sum;
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (tid >= o) upto += v;
      }
      int before = upto - sum;
      if (before < k && k <= upto) {
        int b = 0;
        while (before + s.hist[top - b] < k) before += s.hist[top - b++];
        s.digit = top - b;
        s.left = s.hist[top - b];
      }
    }
    __syncthreads();
    in_step = s.left;
    const int digit = s.digit;
    __syncthreads();
    return digit;
  };
  return bound_search(low, high, kEnough, count);
}

// put(place, i) for the keys above `least` and the first `equal` of those
// equal to it, in order.
template <int THREADS, typename Key, typename Put>
__device__ __forceinline__ void in_order(SelectState& s, int n, int k,
                                         uint32_t least, int equal, Key key,
                                         Put put) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int gt0 = 0, eq0 = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < n && gt0 + min(eq0, equal) < k; i0 += THREADS) {
    const int i = i0 + threadIdx.x;
    const uint32_t x = i < n ? key(i) : 0;
    const bool gt = i < n && x > least, eq = i < n && x == least;
    const unsigned gts = __ballot_sync(0xffffffffu, gt);
    const unsigned eqs = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) {
      s.gt[warp] = __popc(gts);
      s.eq[warp] = __popc(eqs);
    }
    __syncthreads();
    int gt_at = gt0 + __popc(gts & ((1u << lane) - 1u));
    int eq_at = eq0 + __popc(eqs & ((1u << lane) - 1u));
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) gt_at += s.gt[w], eq_at += s.eq[w];
      gt0 += s.gt[w];
      eq0 += s.eq[w];
    }
    if (gt || (eq && eq_at < equal)) put(gt_at + min(eq_at, equal), i);
    __syncthreads();
  }
}

// Pairs of fp32 in one register.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("sub.rn.f32x2 %0, %1, %2;\n" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}
__device__ __forceinline__ float2 apart(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}

// a + b as the sum of two numbers, x its rounding to fp32 (Knuth's two-sum).
// Of two such sums the larger has the larger x, or the same and the larger y.
__device__ __forceinline__ float2 two_sum(float a, float b) {
  const float x = a + b, part = x - a;
  return make_float2(x, (a - (x - part)) + (b - part));
}
__device__ __forceinline__ float2 add_exactly(float2 a, float2 b) {
  const float2 sum = two_sum(a.x, b.x);
  return two_sum(sum.x, sum.y + (a.y + b.y));
}

template <int AB_TYPE>
__device__ __forceinline__ uint64_t widen(uint32_t w) {
  if constexpr (AB_TYPE == 1)
    return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pair(f.x, f.y);
}

// Σ x·w over a warp: a product of two 16-bit floats is exact in fp32; each
// addition keeps what it rounds off, in a second sum.  (In fp64 this took
// twice the time: two additions a clock and SM.)
//   The second sum rounds too.  A lane has four pairs of sums, of n = D/128
// products each.  The two terms that an addition leaves are 2^-23 of M = Σ |x·w|
// each at most, so the j-th finds a second sum of at most j·2^-22·M, and adding
// two to it rounds off j·2^-45·M: n²·2^-46 of M together, D²·2^-60 (4096 columns:
// 2^-36).  That is if all errors have one sign and M is there from the first
// product on; of random ones the second sum stays near 2^-24, 2^-46 together.
// The seven joins of pairs and lanes leave 2^-46 of M each.
struct ExactSum {
  uint64_t hi[2] = {0, 0}, lo[2] = {0, 0};
  template <int AB_TYPE>
  __device__ __forceinline__ void add(uint4 x, uint4 w) {
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // (h + a·b, its product exact; with back = -part of the two-sum)
      uint64_t &h = hi[j & 1], &l = lo[j & 1];
      const uint64_t a = widen<AB_TYPE>(xs[j]), b = widen<AB_TYPE>(ws[j]);
      const uint64_t sum = fma2(a, b, h), back = sub2(h, sum);
      l = add2(l, sub2(h, add2(sum, back)));
      l = add2(l, fma2(a, b, back));
      h = sum;
    }
  }
};
// size + |x·w|
template <int AB_TYPE>
__device__ __forceinline__ uint64_t add_sizes(uint64_t size, uint4 x, uint4 w) {
  const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    size = add2(size, mul2(widen<AB_TYPE>(xs[j]), widen<AB_TYPE>(ws[j])) &
                          0x7fffffff7fffffffull);
  return size;
}
__device__ __forceinline__ float2 across(float2 v, int o) {
  return make_float2(__shfl_xor_sync(0xffffffffu, v.x, o),
                     __shfl_xor_sync(0xffffffffu, v.y, o));
}

// WORDS rows of W at a time, AHEAD loads of each side by side (a row of W comes
// from far).  measure: with this lane's part of Σ |x·w| of the first.
template <int AB_TYPE, int WORDS, int AHEAD>
__device__ __forceinline__ void exact_dots(const uint16_t* x,
                                           const uint16_t* const (&w)[WORDS],
                                           int n, int lane,
                                           float2 (&v)[WORDS], bool measure,
                                           float& size) {
  bool even = (reinterpret_cast<uintptr_t>(x) & 15u) == 0;
#pragma unroll
  for (int i = 0; i < WORDS; ++i)
    even = even && (reinterpret_cast<uintptr_t>(w[i]) & 15u) == 0;
  ExactSum sum[WORDS];
  uint64_t sizes = 0;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int whole = even ? n & ~7 : 0;
#pragma unroll 1
  for (int c = 8 * lane; c < whole; c += 256 * AHEAD) {
    uint4 b[WORDS][AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int at = c + 256 * j;
#pragma unroll
      for (int i = 0; i < WORDS; ++i)
        b[i][j] =
            at < whole ? *reinterpret_cast<const uint4*>(w[i] + at) : zero;
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {  // (x is near)
      const int at = c + 256 * j;
      const uint4 a =
          at < whole ? *reinterpret_cast<const uint4*>(x + at) : zero;
#pragma unroll
      for (int i = 0; i < WORDS; ++i) sum[i].template add<AB_TYPE>(a, b[i][j]);
      if (measure) sizes = add_sizes<AB_TYPE>(sizes, a, b[0][j]);
    }
  }
#pragma unroll 1
  for (int c = whole + 8 * lane; c < n; c += 256) {
    const uint4 a = read_8(x, c, n, false);
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      const uint4 b = read_8(w[i], c, n, false);
      sum[i].template add<AB_TYPE>(a, b);
      if (i == 0 && measure) sizes = add_sizes<AB_TYPE>(sizes, a, b);
    }
  }
#pragma unroll
  for (int i = 0; i < WORDS; ++i) {
    const float2 h0 = apart(sum[i].hi[0]), h1 = apart(sum[i].hi[1]);
    const float2 l0 = apart(sum[i].lo[0]), l1 = apart(sum[i].lo[1]);
    v[i] = add_exactly(
        add_exactly(two_sum(h0.x, l0.x), two_sum(h0.y, l0.y)),
        add_exactly(two_sum(h1.x, l1.x), two_sum(h1.y, l1.y)));
  }
  if (measure) {  // (an infinite or missing logit has no error)
    const float2 m = apart(sizes);
    if (m.x + m.y < INFINITY) size = m.x + m.y;
  }
  // Halves of the lanes sum halves of the words, down to one: v[0] is that of
  // word lane / (32 / WORDS).
  int o = 16;
#pragma unroll
  for (int n = WORDS / 2; n; n >>= 1, o >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const bool upper = lane & o;
      const float2 mine = upper ? v[n + i] : v[i];
      v[i] = add_exactly(mine, across(upper ? v[i] : v[n + i], o));
    }
#pragma unroll 1
  for (; o; o >>= 1) v[0] = add_exactly(v[0], across(v[0], o));
}

// The logits of words c0 to c0 + WORDS - 1 of k in `ids`, before any rounding.
template <int AB_TYPE, int WORDS, int AHEAD>
__device__ __forceinline__ void exact_logits(const VocabCall& p, long long t,
                                             const float* z, const int* ids,
                                             int c0, int k, int lane,
                                             float2* value, bool measure,
                                             float& size) {
  const uint16_t* w[WORDS];
  float2 v[WORDS];
#pragma unroll
  for (int i = 0; i < WORDS; ++i)  // (past the end, the last again)
    w[i] = static_cast<const uint16_t*>(p.W) + ids[min(c0 + i, k - 1)] * p.ldw;
  exact_dots<AB_TYPE, WORDS, AHEAD>(
      static_cast<const uint16_t*>(p.X) + t * p.ldx, w, p.D, lane, v, measure,
      size);
  const int c = c0 + lane / (32 / WORDS);
  if (lane % (32 / WORDS) == 0 && c < k) {
    // (an infinity has no remainder; a NaN is ranked last)
    if (!(fabsf(v[0].x) < INFINITY)) v[0] = make_float2(z[ids[c]], 0.f);
    if (v[0].x != v[0].x) v[0].x = -INFINITY;
    value[c] = v[0];
  }
}

// The first of k words, by value and id.  Their log probabilities are those of
// the fp32 logits, as the given word's is: S is made of them, and what the
// tensor cores drop, towards 0, shrinks both (exact logits beside it were up to
// 1.8 times as far off as fp32 sums that round to nearest).
template <int THREADS>
__device__ __forceinline__ void write_ranked(const VocabCall& p, long long t,
                                             const float* z, const int* ids,
                                             const float2* value, int k,
                                             int thread, float m,
                                             float log_sum) {
  for (int c = thread; c < k; c += THREADS) {
    const float2 v = value[c];
    const int id = ids[c];
    const float logit = z[id];
    int rank = 0;
#pragma unroll 4
    for (int o = 0; o < k; ++o) {
      const float2 w = value[o];
      // (an id twice, where the products gave up: by its place, so that every
      // rank is some word's and every result is written)
      rank += w.x > v.x ||
              (w.x == v.x &&
               (w.y > v.y ||
                (w.y == v.y && (ids[o] < id || (ids[o] == id && o < c)))));
    }
    if (rank < p.alternatives) {
      p.top_out[t * p.alternatives + rank] = id;
      p.top_logp[t * p.alternatives + rank] =
          vocab_log_prob(p, logit, m, log_sum);
    }
  }
}

// A row a block: its results, and its likeliest words.
template <int AB_TYPE, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
    top_kernel(const __grid_constant__ VocabCall p, int row0) {
  constexpr int kWarps = THREADS / 32;
  __shared__ SelectState s;
  __shared__ Stat s_stat[kWarps];
  __shared__ uint2 s_range[kWarps];
  // of the stretches, then candidates; then the values of many candidates
  __shared__ __align__(16) uint32_t s_key[kHeldKeys];
  __shared__ int s_stretch[kStretches], s_id[kMostRanked];
  __shared__ int s_candidate[kCandidates], s_stretches, s_count;
  __shared__ uint32_t s_last, s_size;
  __shared__ float2 s_value[kMostRanked];
  static_assert(2 * kCandidates <= kHeldKeys, "candidates' values");
  griddep_wait();
  griddep_launch_dependents();
  const int learnt = p.header ? p.header->learnt : p.T;
  const int wide = p.header ? p.header->wide : p.wide;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = row0 + blockIdx.x;
  if (r >= learnt) return;
  const long long t = learnt != p.T ? p.token[r] : r;
  if (!p.header && !vocab_is_learnt(p, t)) {
    if (tid == 0) {
      store_results(p, t, r, false, Stat{0.f, 1.f, 0.f}, 0.f, 0.f);
      vocab_unscored(p, t);
    }
    return;
  }
  const int bits = 30 - __clz(wide), half = 1 << bits;  // a stretch
  const int parts = (int)((2ll * p.V + wide - 1) / wide);
  const int k = min(p.alternatives + kSpare, p.V);
  const float* z = p.logits + (long long)blockIdx.x * p.ld_logits;
  if (tid == 0) {
    s_stretches = s_count = 0;
    s_last = s_size = 0;
  }
  // (where the products gave up, maxima and logits need not belong together, and
  // fewer than k elements may reach the bound: what is missing is word 0)
  for (int c = tid; c < k; c += THREADS) s_id[c] = 0;

  // the statistics, and the stretches' maxima
  const bool held = parts <= kHeldKeys;
  uint32_t low = 0xffffffffu, high = 0;
  Stat st = share_of(p, r, tid, parts, THREADS, [&](int g, float z) {
    const uint32_t x = order_of(z);
    if (held) s_key[g] = x;
    low = min(low, x);
    high = max(high, x);
  });
  st = merge_warp(st);
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  if (lane == 0) {
    s_stat[warp] = st;
    s_range[warp] = make_uint2(low, high);
  }
  __syncthreads();
  st = Stat{-INFINITY, 0.f, 0.f};
  if (lane < kWarps) {
    st = s_stat[lane];
    low = s_range[lane].x;
    high = s_range[lane].y;
  }
  st = merge_warp(st);
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  // (in every thread as the first has it)
  st.m = __shfl_sync(0xffffffffu, st.m, 0);
  const float log_sum = logf(__shfl_sync(0xffffffffu, st.s, 0));
  if (tid == 0) store_results(p, t, r, true, st, log_sum, p.picked[r]);

  auto maximum = [&](int g) {
    return held ? s_key[g] : order_of(p.sums[(long long)r * parts + g].w);
  };
  auto logit = [&](int v) -> uint32_t {  // past the vocabulary below all others
    const float* at = z + min(v, p.V - 1);
    float f = 0.f;
    if (span_ok(at, 4, p.logits, 4ll * p.chunk * p.ld_logits, p.status))
      f = *at;
    return v < p.V ? order_of(f) : 0u;
  };
  auto candidate = [&](int v, uint32_t x) {
    const int at = atomicAdd(&s_count, 1);
    if (at < kCandidates) {
      s_key[at] = x;
      s_candidate[at] = v;
    }
  };
  auto largest = [&](int g) {  // (where what is held of them is gone)
    return order_of(p.sums[(long long)r * parts + g].w);
  };
  // A bound that k elements reach: one that k maxima reach, or elements where
  // there are fewer stretches.  Little more than k reach it, unless many are
  // equal.
  bool few;
  if (parts > k) {
    const uint32_t least =
        reached_by<THREADS>(s, parts, k, low, high, maximum);
    for (int g = tid; g < parts; g += THREADS)
      if (maximum(g) >= least) {
        const int at = atomicAdd(&s_stretches, 1);
        if (at < kStretches) s_stretch[at] = g;
      }
    __syncthreads();
    const int stretches = s_stretches;
    few = stretches <= kStretches;
    if (few) {
      // (128 columns a warp at a time, of one stretch or of several narrow
      // ones, and of four such runs side by side)
      const int per = 128 >> bits, sub = lane >> (bits - 2);
      const int in = 4 * (lane & ((half >> 2) - 1));
      const int runs = (stretches + per - 1) / per;
#pragma unroll 1
      for (int i = warp; i < runs; i += 4 * kWarps) {
        float4 f[4];
        int v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int at = (i + j * kWarps) * per + sub;
          v[j] = (s_stretch[min(at, stretches - 1)] << bits) + in;
          const float* from = z + min(v[j], (p.V - 1) & ~3);
          f[j] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i + j * kWarps < runs &&
              span_ok(from, 16, p.logits, 4ll * p.chunk * p.ld_logits,
                      p.status))
            f[j] = *reinterpret_cast<const float4*>(from);
          if (at >= stretches) v[j] = p.V;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float g[4] = {f[j].x, f[j].y, f[j].z, f[j].w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t x = order_of(g[q]);
            if (x >= least && v[j] + q < p.V) candidate(v[j] + q, x);
          }
        }
      }
    }
  } else {
    const uint32_t least =
        reached_by<THREADS>(s, p.V, k, kLowest, high, logit);
#pragma unroll 4
    for (int v = tid; v < p.V; v += THREADS) {
      const uint32_t x = logit(v);
      if (x >= least) candidate(v, x);
    }
    few = true;
  }
  __syncthreads();
  const int count = s_count;
  few = few && count <= kCandidates;
  if (few) {
    for (int c = tid; c < count; c += THREADS) {
      const uint32_t x = s_key[c];
      const int id = s_candidate[c];
      int rank = 0;
#pragma unroll 4
      for (int o = 0; o < count; ++o)
        rank += s_key[o] > x || (s_key[o] == x && s_candidate[o] < id);
      if (rank < k) s_id[rank] = id;
      if (rank == k - 1) s_last = x;
    }
  } else {
    // Many are equal: the k first stretches, in order, and of their elements
    // the k first.
    int stretches = parts, equal;
    __syncthreads();
    if (parts > k) {
      stretches = k;
      const uint32_t least =
          kth_largest<THREADS>(s, parts, k, largest, equal);
      in_order<THREADS>(s, parts, k, least, equal, largest,
                        [&](int at, int g) { s_stretch[at] = g; });
    } else {
      for (int g = tid; g < parts; g += THREADS) s_stretch[g] = g;
      __syncthreads();
    }
    const int n = stretches << bits;
    auto column = [&](int i) {
      return (s_stretch[i >> bits] << bits) + (i & (half - 1));
    };
    auto element = [&](int i) { return logit(column(i)); };
    const uint32_t least = kth_largest<THREADS>(s, n, k, element, equal);
    in_order<THREADS>(s, n, k, least, equal, element,
                      [&](int at, int i) { s_id[at] = column(i); });
    if (tid == 0) s_last = least;
  }
  __syncthreads();

  // ranked by their values before any rounding
  // (many rows: two words a warp, which share x; few: one, with more of it
  // side by side)
  constexpr int kWords = THREADS == 1024 ? 1 : 2;
  constexpr int kAhead = kWords == 1 ? 4 : 2;
  const int* ids = s_id;
  float2* values = s_value;
  int n = k;
  float size = 0.f;
  for (bool first = true;; first = false) {
    // (of a warp's first word the sum of its terms' magnitudes too: of all words
    // it took 22 us more, 1024 tokens, 100000 × 2048, 64 words; this and what
    // follows 8 us of 405, and 3 to 6 of 255, 4096 tokens, 32000 × 768, 5 words)
#pragma unroll 1
    for (int c0 = warp * kWords; c0 < n; c0 += kWarps * kWords)
      exact_logits<AB_TYPE, kWords, kAhead>(
          p, t, z, ids, c0, n, lane, values, first && c0 < kWarps * kWords,
          size);
    if (!first) {
      __syncthreads();
      break;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) size += __shfl_xor_sync(0xffffffffu, size, o);
    if (lane == 0) atomicMax(&s_size, __float_as_uint(size));  // (size >= 0)
    __syncthreads();

    // Words of smaller logits than all of these, but not by more than those may
    // be off: every word that may belong to the first is ranked.
    uint32_t lowest = 0xffffffffu;
    for (int c = lane; c < p.alternatives; c += 32)
      lowest = min(lowest, order_of(s_value[c].x));
    lowest = __reduce_min_sync(0xffffffffu, lowest);
    const float error = logit_error(p.D) * __uint_as_float(s_size);
    const uint32_t need = order_of(reference_of(lowest) - error);
    if (k == p.V || !(error > 0.f) || lowest == kLowest || need > s_last) break;
    if (tid == 0) s_count = 0;
    __syncthreads();
    for (int g = warp; g < parts; g += kWarps) {
      if (largest(g) < need) continue;
#pragma unroll 1
      for (int i = lane; i < half; i += 32) {
        const int v = (g << bits) + i;
        const uint32_t x = logit(v);
        if (x >= need) candidate(v, x);
      }
    }
    __syncthreads();
    const int count = s_count;
    if (count < p.alternatives || count > kCandidates) break;
    __syncthreads();  // (the keys make room for the values)
    n = count;
    ids = s_candidate;
    values = reinterpret_cast<float2*>(s_key);
  }
  write_ranked<THREADS>(p, t, z, ids, values, n, tid, st.m, log_sum);
}

// ------------------------------------------------------------- gradients
// G of a piece's columns, in the rows of the learnt tokens, with zeros up to
// the multiples of 64 that its products sum over; of few tokens in two parts
// (VocabHeader::lo).  Of the first piece, with what the later ones need of
// each row.
constexpr int kGThreads = 256;

template <int AB_TYPE>
__global__ void __launch_bounds__(kGThreads)
    score_g_kernel(const __grid_constant__ VocabCall p, int piece) {
  griddep_wait();
  griddep_launch_dependents();
  const VocabHeader* h = p.header;
  const int learnt = h->learnt, lo = h->lo;
  const int rows = lo ? lo : (learnt + 63) / 64 * 64;
  const int v0 = piece * p.piece, cols = min(p.piece, p.V - v0);
  const int all = (cols + 63) / 64 * 64;
  const int runs = (all + kVocabGRun - 1) / kVocabGRun;
  uint16_t* G = static_cast<uint16_t*>(p.G) +
                (long long)(piece & 1) * p.g_rows * p.piece;
  const int lane = threadIdx.x & 31;
  const long long first =
      (long long)blockIdx.x * (kGThreads / 32) + (threadIdx.x >> 5);
#pragma unroll 1
  for (long long u = first; u < (long long)rows * runs;
       u += (long long)gridDim.x * (kGThreads / 32)) {
    const int r = (int)(u / runs), run = (int)(u - (long long)r * runs);
    score_g_run<AB_TYPE>(
        p, G, r, run * kVocabGRun, v0, cols, all, lo, r < learnt, lane,
        [&](float4& of, int& goal) {
          const long long t = learnt != p.T ? p.token[r] : r;
          of = score_terms(p, t);
          goal = (int)p.targets[t];
          if (run == 0 && piece == 0 && lane == 0) {
            p.terms[r] = of;
            p.goals[r] = goal;
          }
        });
  }
}

}  // namespace

cudaError_t vocab_score_results(const VocabCall& c, int phase, int sms,
                                cudaStream_t stream) {
  const int row0 = phase * c.chunk, rows = std::min(c.chunk, c.T - row0);
  auto launch = [&](auto* fn, int threads) {
    return launch_pdl(fn, dim3(rows), dim3(threads), 0, stream, c, row0);
  };
  if (c.alternatives == 0) return launch(finish_score_kernel, kFinishThreads);
  // A block's warps each sum words' exact logits.  As many as leave every row a
  // place on an SM (1024 threads of 64 registers are all of one): with a row
  // to an SM nothing else hides the wait for rows of W.  32 warps up to a row
  // an SM; 16 up to two (256 tokens, 32000 × 768, 5 words: 41 us with 32, 35
  // with 8, 33 with 16); 8 up to five (400 tokens, 100000 × 2048, 64 words: 223
  // us, 267 with 4; 512 tokens 268 with 32); 4 beyond, of which more blocks
  // overlap (4096 tokens, 32000 × 768, 5 words: 268 us with 8, 246 with 4).
  auto pick = [&](auto bf16, auto f16, int threads) {
    return launch(c.type == GEMM_F32_MIXED_BF16 ? bf16 : f16, threads);
  };
  if (rows <= sms)
    return pick(top_kernel<1, 1024>, top_kernel<0, 1024>, 1024);
  if (rows <= 2 * sms)
    return pick(top_kernel<1, 512>, top_kernel<0, 512>, 512);
  if (rows <= 5 * sms) return pick(top_kernel<1, 256>, top_kernel<0, 256>, 256);
  return pick(top_kernel<1, 128>, top_kernel<0, 128>, 128);
}

cudaError_t vocab_score_g(const VocabCall& c, int piece, int sms,
                          cudaStream_t stream) {
  const int64_t cols = std::min(c.piece, c.V - piece * c.piece);
  const int64_t rows = (c.T + 63) / 64 * 64;
  const int64_t units = rows * ((cols + kVocabGRun - 1) / kVocabGRun);
  const unsigned blocks = (unsigned)std::min<int64_t>(
      (units + kGThreads / 32 - 1) / (kGThreads / 32), 8ll * sms);
  return c.type == GEMM_F32_MIXED_BF16
             ? launch_pdl(score_g_kernel<1>, dim3(blocks), dim3(kGThreads), 0,
                          stream, c, piece)
             : launch_pdl(score_g_kernel<0>, dim3(blocks), dim3(kGThreads), 0,
                          stream, c, piece);
}

}  // namespace gemm_f32_impl
