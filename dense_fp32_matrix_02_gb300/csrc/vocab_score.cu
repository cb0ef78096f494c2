// Log probabilities of given words, entropy and the likeliest words: what
// surrounds their products (vocab_gemm.cu).
//
// With z = X·Wᵀ, c = log2 e / τ and, per row, e_v = 2^(c·z_v − r), r = max c·z,
//   S = Σ e_v,  E = Σ e_v·log2 e_v:
//   lse = ln 2·(r + log2 S),   logp = z_y/τ − lse,
//   entropy = −Σ p·log p = ln 2·(log2 S − E/S).
// The products leave S, E, r and the largest z of each half tile.
//
// The likeliest words.  The k largest elements of a row lie in the k stretches
// (half tiles) with the largest maxima, of equal ones the first: any element
// elsewhere has k larger ones before it, or equal ones with lower ids.  So the
// logits are stored, of some tokens at a time, and of each row only those
// stretches are read, k·128 of V logits.  Storing costs the products nothing
// where they are bound by the tensor cores, and 2·T/D of the weights' bytes
// where they are bound by those.
//   The rank of two logits should not hang on how a sum rounds (on the tile it
// was made in, so on the batch): the k + kSpare largest are computed again
// from the operands, products exact in fp32, summed in pairs of fp32 (48
// bits), and ranked by that.
//
// Gradients.  G = (a·([v = y] − p) − b·p·(log p + H))/τ from the kept logits,
// one pass bound by memory (4 bytes read and 2 written an element), a piece of
// the vocabulary at a time, which then is in L2 for the products.  Making the
// logits again would cost 2·D operations an element instead.
#include <algorithm>

#include "gemm_f32.h"
#include "kernels.h"
#include "vocab.cuh"

namespace gemm_f32_impl {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718056f;

// ------------------------------------------------------------- statistics
struct Stat {
  float m, s, e;  // r, S, E
};

// What a statistic with the reference m counts for beside one of reference
// `ref`: its logarithms move by d.  (Of nothing: d finite, 0 · d = 0.)
__device__ __forceinline__ float moved(float m, float ref) {
  return fmaxf(m - ref, -1e30f);
}

__device__ __forceinline__ Stat merge(Stat a, Stat b) {
  const float m = fmaxf(a.m, b.m);
  const float ref = m == -INFINITY ? 0.f : m;
  const float da = moved(a.m, ref), db = moved(b.m, ref);
  const float ka = exp2f(da), kb = exp2f(db);
  return Stat{m, a.s * ka + b.s * kb,
              ka * (a.e + da * a.s) + kb * (b.e + db * b.s)};
}

__device__ __forceinline__ Stat merge_over(Stat st, int from) {
  for (int o = from; o < 32; o <<= 1) {
    Stat b;
    b.m = __shfl_xor_sync(0xffffffffu, st.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, st.s, o);
    b.e = __shfl_xor_sync(0xffffffffu, st.e, o);
    st = merge(st, b);
  }
  return st;
}

// logp, lse and entropy of the rows from row0 on: 8 rows a block, blockDim / 8
// threads a row that share out its statistics and join them in a fixed order.
__global__ void __launch_bounds__(1024)
    finish_score_kernel(const __grid_constant__ VocabCall p, int row0) {
  __shared__ Stat s_part[32][8];
  griddep_wait();
  griddep_launch_dependents();
  const int learnt = p.header ? p.header->learnt : p.T;
  const int wide = p.header ? p.header->wide : p.wide;
  const int parts = (int)((2ll * p.V + wide - 1) / wide);  // half tiles
  const int in = blockIdx.x * 8 + (threadIdx.x & 7), r = row0 + in;
  const int slice = threadIdx.x >> 3, warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const bool here = in < p.chunk && r < learnt;
  long long t = r;
  bool scored = here;
  float at = 0.f;
  if (warp == 0 && here) {  // ahead of the statistics' loads
    if (learnt != p.T) t = p.token[r];
    if (!p.header) scored = vocab_is_learnt(p, t);
    if (scored) at = p.picked[r];
  }
  // This thread's share, with what each addition rounds off kept (a large
  // vocabulary is many additions).
  Stat st = {-INFINITY, 0.f, 0.f};
  float lost = 0.f, lost_e = 0.f;
  if (here) {
#pragma unroll 4
    for (int g = slice; g < parts; g += blockDim.x >> 3) {
      const long long i = (long long)g * learnt + r;
      const float2 b = p.stats[i];
      const float be = p.slants[i].x;
      const float m = fmaxf(st.m, b.x);
      const float ref = m == -INFINITY ? 0.f : m;
      const float da = moved(st.m, ref), db = moved(b.x, ref);
      const float ka = exp2f(da), kb = exp2f(db);
      const float was = st.s * ka, was_e = ka * (st.e + da * st.s);
      const float more = b.y * kb - lost * ka;
      const float more_e = kb * (be + db * b.y) - lost_e * ka;
      st = Stat{m, was + more, was_e + more_e};
      lost = (st.s - was) - more;
      lost_e = (st.e - was_e) - more_e;
    }
  }
  st = merge_over(st, 8);
  const int warps = blockDim.x >> 5;
  if (warps > 1) {
    if (lane < 8) s_part[warp][lane] = st;
    __syncthreads();
    if (warp > 0) return;
    st = Stat{-INFINITY, 0.f, 0.f};
    for (int w = lane >> 3; w < warps; w += 4)
      st = merge(st, s_part[w][lane & 7]);
    st = merge_over(st, 8);
  }
  if (!here || lane >= 8) return;
  const float log_sum = logf(st.s), l = st.m * kLn2 + log_sum;
  p.loss[t] = scored ? at - l : 0.f;
  p.lse_out[t] = scored ? l : 0.f;
  // (the difference of equal numbers where one word has all: not below 0)
  const float entropy = log_sum - kLn2 * (st.e / st.s);
  p.entropy_out[t] = scored && !(entropy < 0.f) ? entropy : 0.f;
}

// ------------------------------------------------------- likeliest words
constexpr int kTopThreads = 256;
constexpr int kSpare = 8;       // ranked beyond those asked for
constexpr int kMostRanked = kVocabMaxTop + kSpare;
constexpr int kCandidates = 1024;
constexpr int kHeldKeys = 2048;

// Numbers in the order of the floats, from kLowest on; a NaN counts as -Inf.
constexpr uint32_t kLowest = 0x007fffffu;
__device__ __forceinline__ uint32_t order_of(float f) {
  if (f != f) return kLowest;
  const uint32_t u = __float_as_uint(f + 0.f);  // (-0 as 0)
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct SelectState {
  int hist[256];
  int digit, left;
  int gt[kTopThreads / 32], eq[kTopThreads / 32];
};

// The k-th largest of n >= k keys, and how many of those equal to it are
// among the k: the digits of its number, 8 bits at a time, from a histogram of
// the keys that begin as it does.
template <typename Key>
__device__ __forceinline__ uint32_t kth_largest(SelectState& s, int n, int k,
                                                Key key, int& equal) {
  uint32_t prefix = 0;
  int left = k;
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    s.hist[threadIdx.x] = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kTopThreads) {
      const uint32_t x = key(i);
      if (shift == 24 || (x ^ prefix) >> (shift + 8) == 0)
        atomicAdd(&s.hist[(x >> shift) & 255], 1);
    }
    __syncthreads();
    if (threadIdx.x < 32) {  // 8 bins a lane, the largest first
      const int top = 255 - 8 * (int)threadIdx.x;
      int sum = 0;
#pragma unroll
      for (int b = 0; b < 8; ++b) sum += s.hist[top - b];
      int upto = sum;
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if ((int)threadIdx.x >= o) upto += v;
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

// put(place, i) for the keys above `least` and the first `equal` of those
// equal to it, in order.
template <typename Key, typename Put>
__device__ __forceinline__ void in_order(SelectState& s, int n, int k,
                                         uint32_t least, int equal, Key key,
                                         Put put) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int gt0 = 0, eq0 = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < n && gt0 + min(eq0, equal) < k; i0 += kTopThreads) {
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
    for (int w = 0; w < kTopThreads / 32; ++w) {
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
__device__ __forceinline__ double both(uint64_t v) {
  float a, b;
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(v));
  return (double)a + (double)b;
}

template <int AB_TYPE>
__device__ __forceinline__ uint64_t widen(uint32_t w) {
  if constexpr (AB_TYPE == 1)
    return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pair(f.x, f.y);
}

// Σ x·w over a warp: a product of two 16-bit floats is exact in fp32; each
// addition keeps what it rounds off (Knuth's two-sum), in a second sum.
template <int AB_TYPE>
__device__ __forceinline__ double exact_dot(const uint16_t* x, const uint16_t* w,
                                            int n, int lane) {
  const bool vx = (reinterpret_cast<uintptr_t>(x) & 15u) == 0;
  const bool vw = (reinterpret_cast<uintptr_t>(w) & 15u) == 0;
  uint64_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll 2
  for (int c = 8 * lane; c < n; c += 256) {
    const uint4 a = read_8(x, c, n, vx), b = read_8(w, c, n, vw);
    const uint32_t av[4] = {a.x, a.y, a.z, a.w};
    const uint32_t bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint64_t &h = hi[j & 1], &l = lo[j & 1];
      const uint64_t term = mul2(widen<AB_TYPE>(av[j]), widen<AB_TYPE>(bv[j]));
      const uint64_t sum = add2(h, term), part = sub2(sum, h);
      l = add2(l, add2(sub2(h, sub2(sum, part)), sub2(term, part)));
      h = sum;
    }
  }
  double v = (both(hi[0]) + both(hi[1])) + (both(lo[0]) + both(lo[1]));
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A row a block.
template <int AB_TYPE>
__global__ void __launch_bounds__(kTopThreads)
    top_kernel(const __grid_constant__ VocabCall p, int row0) {
  __shared__ SelectState s;
  __shared__ uint32_t s_key[kHeldKeys];  // of the stretches, then candidates
  __shared__ int s_stretch[kMostRanked], s_id[kMostRanked];
  __shared__ int s_candidate[kCandidates], s_count;
  __shared__ double s_value[kMostRanked];
  static_assert(kCandidates <= kHeldKeys, "candidates' keys");
  griddep_wait();
  griddep_launch_dependents();
  const int learnt = p.header ? p.header->learnt : p.T;
  const int wide = p.header ? p.header->wide : p.wide;
  const int r = row0 + blockIdx.x;
  if (r >= learnt) return;
  const long long t = learnt != p.T ? p.token[r] : r;
  if (!p.header && !vocab_is_learnt(p, t)) {
    if (threadIdx.x == 0) vocab_unscored(p, t);
    return;
  }
  const int bits = 30 - __clz(wide), half = 1 << bits;  // a stretch
  const int parts = (int)((2ll * p.V + wide - 1) / wide);
  const int k = min(p.alternatives + kSpare, p.V);
  const float* z = p.logits + (long long)blockIdx.x * p.ld_logits;
  const int tid = threadIdx.x;

  // the stretches
  uint32_t least = 0;
  int stretches = parts;
  if (parts > k) {
    auto maximum = [&](int g) {
      return order_of(p.slants[(long long)g * learnt + r].y);
    };
    const bool held = parts <= kHeldKeys;
    if (held) {
#pragma unroll 4
      for (int g = tid; g < parts; g += kTopThreads) s_key[g] = maximum(g);
      __syncthreads();
    }
    auto key = [&](int g) { return held ? s_key[g] : maximum(g); };
    int equal;
    least = kth_largest(s, parts, k, key, equal);
    in_order(s, parts, k, least, equal, key,
             [&](int at, int g) { s_stretch[at] = g; });
    stretches = k;
  } else {
    for (int g = tid; g < parts; g += kTopThreads) s_stretch[g] = g;
  }
  if (tid == 0) s_count = 0;
  __syncthreads();

  // Their elements; past the vocabulary none, which no k elements need.
  const int n = stretches << bits;
  auto column = [&](int i) {
    return (s_stretch[i >> bits] << bits) + (i & (half - 1));
  };
  auto key = [&](int i) -> uint32_t {
    const int v = column(i);
    return v < p.V &&
                   span_ok(z + v, 4, p.logits, 4ll * p.chunk * p.ld_logits,
                           p.status)
               ? order_of(z[v])
               : 0u;
  };
  // Those that the smallest of the maxima leaves are few, unless many are
  // equal or the stretches are all there are.
  bool few = parts > k;
  if (few) {
#pragma unroll 4
    for (int i = tid; i < n; i += kTopThreads) {
      const uint32_t x = key(i);
      if (x >= least) {
        const int at = atomicAdd(&s_count, 1);
        if (at < kCandidates) {
          s_key[at] = x;
          s_candidate[at] = column(i);
        }
      }
    }
    __syncthreads();
    few = s_count <= kCandidates;
  }
  if (few) {
    const int count = s_count;
    for (int c = tid; c < count; c += kTopThreads) {
      const uint32_t x = s_key[c];
      const int id = s_candidate[c];
      int rank = 0;
      for (int o = 0; o < count; ++o)
        rank += s_key[o] > x || (s_key[o] == x && s_candidate[o] < id);
      if (rank < k) s_id[rank] = id;
    }
  } else {
    int equal;
    least = kth_largest(s, n, k, key, equal);
    in_order(s, n, k, least, equal, key,
             [&](int at, int i) { s_id[at] = column(i); });
  }
  __syncthreads();

  // ranked by their values before any rounding
  const uint16_t* x = static_cast<const uint16_t*>(p.X) + t * p.ldx;
  for (int c = tid >> 5; c < k; c += kTopThreads / 32) {
    const int id = s_id[c];
    double v = exact_dot<AB_TYPE>(
        x, static_cast<const uint16_t*>(p.W) + id * p.ldw, p.D, tid & 31);
    if (v != v) v = z[id];  // (infinities: the sum's, not of what it rounds off)
    if (v != v) v = -INFINITY;
    if ((tid & 31) == 0) s_value[c] = v;
  }
  __syncthreads();
  for (int c = tid; c < k; c += kTopThreads) {
    const double v = s_value[c];
    const int id = s_id[c];
    int rank = 0;
    for (int o = 0; o < k; ++o)
      rank += s_value[o] > v || (s_value[o] == v && s_id[o] < id);
    if (rank < p.alternatives) {
      p.top_out[t * p.alternatives + rank] = id;
      p.top_logp[t * p.alternatives + rank] =
          (float)(v / (double)p.tau - (double)p.lse_out[t]);
    }
  }
}

// ------------------------------------------------------------- gradients
constexpr int kGThreads = 256, kGColumns = 16 * kGThreads;

// G of a piece's columns, in the rows of the learnt tokens, with zeros up to
// the multiples of 64 that its products sum over; of few tokens in two parts
// (VocabHeader::lo).  With p = 2^t, t = z·c − lse·log2 e,
//   G = p·(A + B·t) + [v = y]·a,  A = −(a + b·H),  B = −b·ln 2
// (a, b: times 1/τ and the scale of G).
template <int AB_TYPE>
__global__ void __launch_bounds__(kGThreads)
    score_g_kernel(const __grid_constant__ VocabCall p, int piece) {
  griddep_wait();
  griddep_launch_dependents();
  const VocabHeader* h = p.header;
  const int learnt = h->learnt, lo = h->lo;
  const int rows = lo ? lo : (learnt + 63) / 64 * 64;
  const int v0 = piece * p.piece, cols = min(p.piece, p.V - v0);
  const int all = (cols + 63) / 64 * 64, segments = (all + kGColumns - 1) / kGColumns;
  const float c2 = p.inv_tau * kLog2e, scale = h->scale * p.inv_tau;
  uint16_t* G = static_cast<uint16_t*>(p.G) +
                (long long)(piece & 1) * p.g_rows * p.piece;
  const long long extent = 2ll * p.g_rows * p.piece;
#pragma unroll 1
  for (long long u = blockIdx.x; u < (long long)rows * segments;
       u += gridDim.x) {
    const int r = (int)(u / segments), seg = (int)(u - (long long)r * segments);
    float A = 0.f, B = 0.f, a = 0.f, shift = 0.f;
    int target = -1;
    const bool here = r < learnt;
    if (here) {
      const long long t = learnt != p.T ? p.token[r] : r;
      const float entropy = p.entropy[t];
      a = p.grad_loss[t * p.grad_stride] * scale;
      const float b =
          p.grad_entropy ? p.grad_entropy[t * p.entropy_stride] * scale : 0.f;
      A = -(a + b * entropy);
      B = -b * kLn2;
      shift = -p.lse[t] * kLog2e;
      target = (int)p.targets[t] - v0;
    }
    const float* z = p.logits + (long long)r * p.ld_logits + v0;
    const int c0 = seg * kGColumns + 8 * threadIdx.x;
    float f[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = c0 + 8 * kGThreads * i;
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
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = c0 + 8 * kGThreads * i;
      if (c >= all) break;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = fmaf(f[i][j], c2, shift), e = exp2_fast(t);
        // (2^-200 is 0: an infinity's product with it would not be)
        const float g = e * fmaf(B, fmaxf(t, -200.f), A);
        f[i][j] = here && c + j < cols ? g : 0.f;
      }
      if (target >= c && target < c + 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (target == c + j) f[i][j] += a;
      }
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = pack16<AB_TYPE>(f[i][2 * j], f[i][2 * j + 1]);
      uint16_t* to = G + (long long)r * p.piece + c;
      if (!span_ok(to, 16, p.G, (p.pieces > 1 ? 2 : 1) * extent, p.status))
        continue;
      *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
      if (!lo) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = pack16_rest<AB_TYPE>(f[i][2 * j], f[i][2 * j + 1], w[j]);
      to += (long long)lo * p.piece;
      if (span_ok(to, 16, p.G, (p.pieces > 1 ? 2 : 1) * extent, p.status))
        *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

}  // namespace

cudaError_t vocab_score_results(const VocabCall& c, int phase, int sms,
                                cudaStream_t stream) {
  const int row0 = phase * c.chunk, rows = std::min(c.chunk, c.T - row0);
  // a thread's share of a row: a few statistics
  const int parts = (c.V + 127) / 128;
  const int threads = parts <= 16 ? 32 : parts <= 128 ? 256 : 1024;
  cudaError_t e = launch_pdl(finish_score_kernel, dim3((rows + 7) / 8),
                             dim3(threads), 0, stream, c, row0);
  if (e != cudaSuccess || c.alternatives == 0) return e;
  return c.type == GEMM_F32_MIXED_BF16
             ? launch_pdl(top_kernel<1>, dim3(rows), dim3(kTopThreads), 0,
                          stream, c, row0)
             : launch_pdl(top_kernel<0>, dim3(rows), dim3(kTopThreads), 0,
                          stream, c, row0);
}

cudaError_t vocab_score_g(const VocabCall& c, int piece, int sms,
                          cudaStream_t stream) {
  const int64_t cols = std::min(c.piece, c.V - piece * c.piece);
  const int64_t rows = (c.T + 63) / 64 * 64;
  const int64_t units = rows * ((cols + kGColumns - 1) / kGColumns);
  const unsigned blocks = (unsigned)std::min<int64_t>(units, 8ll * sms);
  return c.type == GEMM_F32_MIXED_BF16
             ? launch_pdl(score_g_kernel<1>, dim3(blocks), dim3(kGThreads), 0,
                          stream, c, piece)
             : launch_pdl(score_g_kernel<0>, dim3(blocks), dim3(kGThreads), 0,
                          stream, c, piece);
}

}  // namespace gemm_f32_impl
