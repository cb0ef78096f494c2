// The global norm of many gradients, and clipping by it (the definitions are
// in include/gemm_f32.h).
//
//   n = sqrt(Σ over every element of every gradient of g²)
//   g ← g·min(1, max_norm / n)
//
// Bound by memory: the factor depends on every element, so a gradient that
// does not stay in L2 is read twice and written once.  Two launches: the
// first writes one partial sum a block, the second has every block add the
// partial sums up (some hundred doubles, in the same order in each) and scales
// its share.  No atomics: the same call gives the same bits.
//
// The list of gradients travels in the kernels' parameters, so that nothing
// is copied to the device and a captured launch holds what it works on.  All
// gradients are one line of 16-byte groups, cut into equal chunks; a block
// takes every gridDim-th chunk and finds its gradient by bisection (chunks of
// 256 KB at most: with 64 KB 1.3e9 elements took 1228 us, with 16 KB 1390).  The
// second launch takes the chunks from the last to the first: what the first read
// last is still in L2 (1e8 elements 110 us, 113 the other way).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <functional>
#include <memory>
#include <new>
#include <type_traits>

#include "gemm_f32.h"
#include "kernels.h"

namespace gemm_f32_impl {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // 16-byte groups a thread loads side by side
constexpr int kLeastChunk = kThreads;               // groups
constexpr int kRun = 4 * kAhead * kThreads;         // summed in fp32: 64 KB
constexpr int kMostChunk = 4 * kRun;
constexpr int kBlocksPerSm = 4;
constexpr int kMaxBlocks = 2048;
// Gradients of a launch: few (1.8 KB of parameters), or many (29 KB); more are
// several launches.
constexpr int kFew = 32, kMany = 520;

// One gradient.  Rows are cut into groups of 16 bytes that start on 16-byte
// boundaries of memory; the first and the last may lie partly outside the row.
struct Entry {
  const char* in;
  char* out;
  long long cols, ld, ld_out;  // elements
  int rows;
  int type;
};

template <int N>
struct List {
  Entry entry[N];
  long long first[N + 1];  // chunks before this launch's gradients
  int n;
  int chunk;               // groups of a chunk
  unsigned int* status;
};

__host__ __device__ constexpr int elements(int type) {
  return type == GEMM_F32_GRAD_F32 ? 4 : 8;  // of a group
}
// Groups of a row: as many as hold it wherever it starts, none partly
// outside where all rows start on a boundary.
__host__ __device__ __forceinline__ long long groups(const Entry& e) {
  const int n = elements(e.type), size = 16 / n;
  const bool even = (reinterpret_cast<uintptr_t>(e.in) & 15u) == 0 &&
                    (e.rows == 1 || e.ld * size % 16 == 0);
  return (e.cols + (even ? n - 1 : 2 * n - 2)) / n;
}

template <int TYPE>
__device__ __forceinline__ void unpack(uint4 v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (TYPE == GEMM_F32_GRAD_F32) {
      f[i] = __uint_as_float(w[i]);
    } else if constexpr (TYPE == GEMM_F32_GRAD_BF16) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
}

template <int TYPE>
__device__ __forceinline__ uint4 pack(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (TYPE == GEMM_F32_GRAD_F32) {
      w[i] = __float_as_uint(f[i]);
    } else if constexpr (TYPE == GEMM_F32_GRAD_BF16) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    } else {
      const __half2 p = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Where a group lies: its row, and its first element's column, which is
// negative in a row that starts off a boundary.
struct Place {
  long long row, col;
  bool here, whole;
};

template <int TYPE>
struct Chunk {
  static constexpr int N = elements(TYPE), SIZE = 16 / N;
  using Bits = typename std::conditional<N == 4, uint32_t, uint16_t>::type;
  const Entry& e;
  long long per, row0, j0;
  int count;  // groups of this chunk

  __device__ __forceinline__ Chunk(const Entry& e_, long long chunk, int size)
      : e(e_), per(groups(e_)) {
    const long long at = chunk * size, all = per * e.rows;
    count = (int)min((long long)size, all - at);
    row0 = e.rows == 1 ? 0 : at / per;
    j0 = at - row0 * per;
  }
  __device__ __forceinline__ Place place(int k) const {
    Place p;
    p.row = row0;
    long long j = j0 + k;
    if (e.rows > 1 && j >= per) {  // (fewer than 2^31 groups: the host checks)
      const unsigned more = (unsigned)j / (unsigned)per;
      p.row += more;
      j -= (long long)more * per;
    }
    const uintptr_t row =
        reinterpret_cast<uintptr_t>(e.in) + p.row * e.ld * SIZE;
    p.col = j * N - (long long)((row & 15u) / SIZE);
    p.here = k < count && p.col < e.cols;
    p.whole = p.here && p.col >= 0 && p.col + N <= e.cols;
    return p;
  }
  __device__ __forceinline__ const Bits* from(const Place& p) const {
    return reinterpret_cast<const Bits*>(e.in) + p.row * e.ld + p.col;
  }
  __device__ __forceinline__ Bits* to(const Place& p) const {
    return reinterpret_cast<Bits*>(e.out) + p.row * e.ld_out + p.col;
  }
  __device__ __forceinline__ uint4 load(const Place& p,
                                        unsigned int* status) const {
    const Bits* from_ = from(p);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (p.whole) {
      if (span_ok(from_, 16, e.in, SIZE * ((e.rows - 1) * e.ld + e.cols),
                  status))
        v = *reinterpret_cast<const uint4*>(from_);
    } else if (p.here) {
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (p.col + i >= 0 && p.col + i < e.cols)
          w[i * SIZE / 4] |= (uint32_t)from_[i] << (i * SIZE % 4 * 8);
      v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return v;
  }
  __device__ __forceinline__ void load_all(const Place (&p)[kAhead],
                                           uint4 (&v)[kAhead],
                                           unsigned int* status) const {
    if (p[0].whole && p[1].whole && p[2].whole && p[3].whole) {
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {  // side by side
        v[a] = make_uint4(0, 0, 0, 0);
        if (span_ok(from(p[a]), 16, e.in, SIZE * ((e.rows - 1) * e.ld + e.cols),
                    status))
          v[a] = *reinterpret_cast<const uint4*>(from(p[a]));
      }
    } else {
#pragma unroll
      for (int a = 0; a < kAhead; ++a) v[a] = load(p[a], status);
    }
  }
  __device__ __forceinline__ void store(const Place& p, uint4 v,
                                        unsigned int* status) const {
    Bits* to_ = to(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const unsigned odd = reinterpret_cast<uintptr_t>(to_) & 15u;
    if (p.whole) {
      if (!span_ok(to_, 16, e.out, SIZE * ((e.rows - 1) * e.ld_out + e.cols),
                   status))
        return;
      if (odd == 0) {
        *reinterpret_cast<uint4*>(to_) = v;
        return;
      }
      if ((odd & 7u) == 0) {
        reinterpret_cast<uint2*>(to_)[0] = make_uint2(v.x, v.y);
        reinterpret_cast<uint2*>(to_)[1] = make_uint2(v.z, v.w);
        return;
      }
      if ((odd & 3u) == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          reinterpret_cast<uint32_t*>(to_)[i] = w[i];
        return;
      }
    }
    if (!p.here) return;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (p.col + i >= 0 && p.col + i < e.cols)
        to_[i] = (Bits)(w[i * SIZE / 4] >> (i * SIZE % 4 * 8));
  }

  // This thread's groups from `first` to before `last`, kAhead at a time.
  template <typename Fn>
  __device__ __forceinline__ void each(int first, int last, Fn fn) const {
#pragma unroll 1
    for (int k0 = first + threadIdx.x; k0 < last; k0 += kAhead * kThreads) {
      Place p[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) p[a] = place(k0 + a * kThreads);
      fn(p);
    }
  }
};

// The squares of a thread's part of a run are summed in fp32 (at most 16
// groups, 128 squares, in 4 sums), the runs in fp64.  Squares that overflow
// fp32, or of which too little is left, show in the sum: those groups are read
// again and summed in fp64, whose range holds them.
template <int TYPE>
__device__ __forceinline__ double sum_run(const Chunk<TYPE>& c, int first,
                                          int last, unsigned int* status) {
  constexpr int N = Chunk<TYPE>::N;
  const Entry& e = c.e;
  float run[4] = {0.f, 0.f, 0.f, 0.f};
  uint32_t any = 0;
  c.each(first, last, [&](const Place(&p)[kAhead]) {
    uint4 v[kAhead];
    c.load_all(p, v, status);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      any |= v[a].x | v[a].y | v[a].z | v[a].w;
      float f[N];
      unpack<TYPE>(v[a], f);
#pragma unroll
      for (int i = 0; i < N; ++i) run[i & 3] = fmaf(f[i], f[i], run[i & 3]);
    }
  });
  const float sum = (run[0] + run[1]) + (run[2] + run[3]);
  // (`any` of the sign bits alone: zeros, read twice)
  if (any != 0 && !(sum >= 0x1p-96f && sum <= 1e37f)) {
    double wide = 0.0;
#pragma unroll 1
    for (int k = first + threadIdx.x; k < last; k += kThreads) {
      float f[N];
      unpack<TYPE>(c.load(c.place(k), status), f);
#pragma unroll
      for (int i = 0; i < N; ++i) wide += (double)f[i] * (double)f[i];
    }
    return wide;
  }
  return sum;
}

template <int TYPE>
__device__ __forceinline__ double sum_chunk(const Entry& e, long long chunk,
                                            int size, unsigned int* status) {
  const Chunk<TYPE> c(e, chunk, size);
  double sum = 0.0;
#pragma unroll 1
  for (int k = 0; k < c.count; k += kRun)
    sum += sum_run<TYPE>(c, k, min(k + kRun, c.count), status);
  return sum;
}

// min(1, max_norm / n) in two parts, hi rounded down, so that a product with it
// rounds once (g·hi + g·lo, its sum in one step and of one sign: a zero keeps
// its own).  A quotient below 2^-60 is kept in fp64: it may be below fp32's
// smallest normal number.
struct Factor {
  float hi, lo;
  double small;  // or 0
  __device__ __forceinline__ bool one() const { return hi == 1.f; }
};
__device__ __forceinline__ Factor factor_of(double n, float max_norm) {
  Factor f = {1.f, 0.f, 0.0};
  if (!(n > (double)max_norm && n < INFINITY)) return f;
  const double q = max_norm / n;
  if (q < 0x1p-60) return Factor{0.f, 0.f, q};
  // (what rounds to 1 moves no fp32 number by more than half a step)
  if ((float)q == 1.f) return f;
  f.hi = __double2float_rd(q);
  f.lo = (float)(q - f.hi);
  return f;
}

template <int TYPE>
__device__ __forceinline__ void scale_chunk(const Entry& e, long long chunk,
                                            int size, const Factor& factor,
                                            unsigned int* status) {
  const Chunk<TYPE> c(e, chunk, size);
  constexpr int N = Chunk<TYPE>::N;
  // factor 1: a copy, of NaN and infinities too
  auto scaled = [&](uint4 v) {
    if (factor.one()) return v;
    float f[N];
    unpack<TYPE>(v, f);
    if (factor.hi > 0.f) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        f[i] = fmaf(f[i], factor.hi, f[i] * factor.lo);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = (float)(f[i] * factor.small);
    }
    return pack<TYPE>(f);
  };
  c.each(0, c.count, [&](const Place(&p)[kAhead]) {
    uint4 v[kAhead];
    c.load_all(p, v, status);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) c.store(p[a], scaled(v[a]), status);
  });
}

// Sums of fp64 take 16 cycles a warp and addition, on one unit an SM: as few
// as can be, by the first warp (every thread of every block adding up the
// partial sums and dividing took 8 us of a call).
__device__ __forceinline__ double warp_sum(double v) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The gradient of a chunk, and the chunk's number in it.
template <int N>
__device__ __forceinline__ int find(const List<N>& list, long long& chunk) {
  int low = 0, high = list.n;  // first[low] <= chunk < first[high]
  while (high - low > 1) {
    const int mid = (low + high) >> 1;
    if (list.first[mid] <= chunk) low = mid; else high = mid;
  }
  chunk -= list.first[low];
  return low;
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    norm_kernel(const __grid_constant__ List<N> list, double* partial) {
  griddep_wait();
  griddep_launch_dependents();
  double sum = 0.0;
#pragma unroll 1
  for (long long i = blockIdx.x; i < list.first[list.n]; i += gridDim.x) {
    long long chunk = i;
    const Entry& e = list.entry[find(list, chunk)];
    if (e.type == GEMM_F32_GRAD_BF16)
      sum += sum_chunk<GEMM_F32_GRAD_BF16>(e, chunk, list.chunk, list.status);
    else if (e.type == GEMM_F32_GRAD_F16)
      sum += sum_chunk<GEMM_F32_GRAD_F16>(e, chunk, list.chunk, list.status);
    else
      sum += sum_chunk<GEMM_F32_GRAD_F32>(e, chunk, list.chunk, list.status);
  }
  __shared__ double part[kThreads];
  part[threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.x >= 32) return;
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) sum += part[threadIdx.x + 32 * w];
  sum = warp_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// The norm from the partial sums, and the gradients times the factor.  A norm
// that is not finite clips nothing.
template <int N>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    clip_kernel(const __grid_constant__ List<N> list, const double* partial,
                int partials, float max_norm, float* norm) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ Factor s_factor;
  if (threadIdx.x < 32) {
    double sum = 0.0;
#pragma unroll 8
    for (int i = threadIdx.x; i < partials; i += 32) sum += partial[i];
    sum = warp_sum(sum);
    if (threadIdx.x == 0) {
      const double n = sqrt(sum);
      if (norm && blockIdx.x == 0) *norm = (float)n;
      s_factor = factor_of(n, max_norm);
    }
  }
  __syncthreads();
  const Factor factor = s_factor;
  const long long last = list.first[list.n] - 1;
#pragma unroll 1
  for (long long i = blockIdx.x; i <= last; i += gridDim.x) {
    long long chunk = last - i;
    const Entry& e = list.entry[find(list, chunk)];
    if (factor.one() && e.in == e.out && e.ld == e.ld_out) continue;
    if (e.type == GEMM_F32_GRAD_BF16)
      scale_chunk<GEMM_F32_GRAD_BF16>(e, chunk, list.chunk, factor,
                                      list.status);
    else if (e.type == GEMM_F32_GRAD_F16)
      scale_chunk<GEMM_F32_GRAD_F16>(e, chunk, list.chunk, factor,
                                     list.status);
    else
      scale_chunk<GEMM_F32_GRAD_F32>(e, chunk, list.chunk, factor,
                                     list.status);
  }
}

// ------------------------------------------------------------- host side
// Elements of a gradient: its bytes and groups stay far inside 64 bits.
constexpr int64_t kMostElements = 1ll << 48;
constexpr int64_t kMostRows = 0x7fffffff;

int check(const gemm_f32_grad& g, bool clip) {
  if (g.type != GEMM_F32_GRAD_BF16 && g.type != GEMM_F32_GRAD_F16 &&
      g.type != GEMM_F32_GRAD_F32)
    return GEMM_F32_ERR_INVALID_ARG;
  if (g.rows < 0 || g.cols < 0) return GEMM_F32_ERR_INVALID_ARG;
  if (g.rows == 0 || g.cols == 0) return GEMM_F32_OK;
  const uintptr_t size = g.type == GEMM_F32_GRAD_F32 ? 4 : 2;
  if (!g.data || (clip && !g.out) ||
      reinterpret_cast<uintptr_t>(g.data) % size ||
      (clip && reinterpret_cast<uintptr_t>(g.out) % size))
    return GEMM_F32_ERR_INVALID_ARG;
  if (g.rows > 1 && (g.ld < g.cols || (clip && g.ld_out < g.cols)))
    return GEMM_F32_ERR_INVALID_ARG;
  if (g.cols > kMostElements / g.rows || g.rows > kMostRows)
    return GEMM_F32_ERR_UNSUPPORTED;
  if (g.rows > 1 && (g.cols > kMostRows || g.ld > kMostElements / g.rows ||
                     (clip && g.ld_out > kMostElements / g.rows)))
    return GEMM_F32_ERR_UNSUPPORTED;
  return GEMM_F32_OK;
}

// Whether two gradients go to the same place (one that is listed twice, as of
// a shared weight, would be scaled twice or once).
bool twice(int64_t n, const gemm_f32_grad* all) {
  if (n < 2) return false;
  std::unique_ptr<const void*[]> to(new (std::nothrow) const void*[n]);
  if (!to) return false;  // (no memory for the check)
  int64_t m = 0;
  for (int64_t i = 0; i < n; ++i)
    if (all[i].rows && all[i].cols) to[m++] = all[i].out;
  std::sort(to.get(), to.get() + m, std::less<const void*>());
  return std::adjacent_find(to.get(), to.get() + m) != to.get() + m;
}

Entry entry(const gemm_f32_grad& g, bool clip) {
  Entry e;
  e.in = static_cast<const char*>(g.data);
  e.out = clip ? static_cast<char*>(g.out) : nullptr;
  e.cols = g.cols, e.rows = (int)g.rows;
  e.ld = g.rows > 1 ? g.ld : g.cols;
  e.ld_out = !clip ? 0 : g.rows > 1 ? g.ld_out : g.cols;
  e.type = (int)g.type;
  // rows one behind the other are one row
  if (e.rows > 1 && e.ld == e.cols && (!clip || e.ld_out == e.cols)) {
    e.cols *= e.rows;
    e.rows = 1;
    e.ld = e.cols;
    if (clip) e.ld_out = e.cols;
  }
  return e;
}

// Launches `go(list, blocks)` for up to N gradients at a time.
template <int N, typename Go>
cudaError_t in_lists(int64_t n, const gemm_f32_grad* all, bool clip, int chunk,
                     int most_blocks, unsigned int* status, Go go) {
  List<N> list;
  list.n = 0, list.first[0] = 0;
  list.chunk = chunk, list.status = status;
  cudaError_t e = cudaSuccess;
  for (int64_t i = 0; i <= n && e == cudaSuccess; ++i) {
    if (i < n && all[i].rows && all[i].cols) {
      list.entry[list.n] = entry(all[i], clip);
      const Entry& x = list.entry[list.n];
      const long long count = groups(x) * x.rows;
      list.first[list.n + 1] =
          list.first[list.n] + (count + chunk - 1) / chunk;
      ++list.n;
    }
    if (list.n == N || (i == n && list.n > 0)) {
      e = go(list, (int)std::min<long long>(list.first[list.n], most_blocks));
      list.n = 0;
    }
  }
  return e;
}

int64_t launches(int64_t n) {
  return n <= kFew ? 1 : (n + kMany - 1) / kMany;
}

int run(int64_t n, const gemm_f32_grad* all, bool clip, float max_norm,
        float* norm, void* ws, int64_t ws_bytes, gemm_f32_stream_t stream_) {
  if (n < 0 || (n > 0 && !all) || !norm || ws_bytes < 0)
    return GEMM_F32_ERR_INVALID_ARG;
  if (n > kMostRows) return GEMM_F32_ERR_UNSUPPORTED;
  if (clip && !(max_norm >= 0.f)) return GEMM_F32_ERR_INVALID_ARG;
  long long total = 0;
  int64_t used = 0;
  for (int64_t i = 0; i < n; ++i) {
    const int st = check(all[i], clip);
    if (st != GEMM_F32_OK) return st;
    if (all[i].rows == 0 || all[i].cols == 0) continue;
    const Entry e = entry(all[i], clip);
    total += groups(e) * e.rows;
    if (total > (1ll << 58)) return GEMM_F32_ERR_UNSUPPORTED;
    ++used;
  }
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 15u) != 0 ||
      ws_bytes < gemm_f32_grad_workspace_size(n))
    return GEMM_F32_ERR_INVALID_ARG;
  if (clip && twice(n, all)) return GEMM_F32_ERR_INVALID_ARG;
  int sms = 0, cc = 0;
  WaitCfg wc;
  cudaError_t e = device_facts(&sms, &cc, &wc);
  if (e != cudaSuccess) return record_cuda_error(e);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const int most = std::min(kBlocksPerSm * sms, kMaxBlocks);
  // the largest chunks of which every block has two, or the least
  int chunk = kLeastChunk;
  while (chunk < kMostChunk && total / (2 * chunk) >= 2ll * most) chunk *= 2;
  double* partial = static_cast<double*>(ws);
  int partials = 0;
  auto sum = [&](const auto& list, int blocks) {
    constexpr int N = sizeof(list.entry) / sizeof(Entry);
    const cudaError_t st = launch_pdl(norm_kernel<N>, dim3(blocks),
                                      dim3(kThreads), 0, stream, list,
                                      partial + partials);
    partials += blocks;
    return st;
  };
  bool told = false;  // the norm is written by the first of these
  auto scale = [&](const auto& list, int blocks) {
    constexpr int N = sizeof(list.entry) / sizeof(Entry);
    const cudaError_t st = launch_pdl(
        clip_kernel<N>, dim3(blocks), dim3(kThreads), 0, stream, list,
        (const double*)partial, partials, max_norm, told ? nullptr : norm);
    told = true;
    return st;
  };
  const bool few = used <= kFew;
  e = few ? in_lists<kFew>(n, all, clip, chunk, most, wc.status, sum)
          : in_lists<kMany>(n, all, clip, chunk, most, wc.status, sum);
  if (e == cudaSuccess && clip)
    e = few ? in_lists<kFew>(n, all, clip, chunk, most, wc.status, scale)
            : in_lists<kMany>(n, all, clip, chunk, most, wc.status, scale);
  if (e == cudaSuccess && !told) {
    List<kFew> none = {};
    e = scale(none, 1);
  }
  return e == cudaSuccess ? GEMM_F32_OK : record_cuda_error(e);
}

}  // namespace
}  // namespace gemm_f32_impl

using namespace gemm_f32_impl;

extern "C" {

int gemm_f32_grad_norm(int64_t n, const gemm_f32_grad* grads, float* norm,
                       void* workspace, int64_t workspace_bytes,
                       gemm_f32_stream_t stream) {
  return run(n, grads, false, 0.f, norm, workspace, workspace_bytes, stream);
}

int gemm_f32_grad_clip(int64_t n, const gemm_f32_grad* grads, float max_norm,
                       float* norm, void* workspace, int64_t workspace_bytes,
                       gemm_f32_stream_t stream) {
  return run(n, grads, true, max_norm, norm, workspace, workspace_bytes,
             stream);
}

int64_t gemm_f32_grad_workspace_size(int64_t n) {
  if (n < 0) return -GEMM_F32_ERR_INVALID_ARG;
  if (n > kMostRows) return -GEMM_F32_ERR_UNSUPPORTED;
  return std::max<int64_t>(launches(n), 1) * kMaxBlocks *
         (int64_t)sizeof(double);
}

}  // extern "C"
