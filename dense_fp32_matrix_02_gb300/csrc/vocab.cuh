// What the vocabulary losses' kernels share: the targets as the kernels see
// them and the state that a call keeps in its workspace.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>

#include "common.cuh"

namespace gemm_f32_impl {

constexpr int kVocabMaxTop = 256;

// Written by the first kernels of a call, read by the later ones.
struct VocabHeader {
  int learnt;       // tokens that are learnt from
  float scale;      // gradients: G is stored times this power of two
  float inv_scale;  // 1 / scale
};

// The target distributions.  Row t of ids and log_q (top entries a row)
// holds token t's entries that count, sorted by id, then INT_MAX; a weight
// is exp(log_q).  Tokens that are learnt from are numbered in order: row r
// of a kernel's matrices is token token[r], and row[t] is r or -1.
struct VocabTargets {
  const VocabHeader* header;
  const int* token;
  const int* row;
  const int* ids;
  const float* log_q;
  int top;
  float inv_tau;
};

__device__ __forceinline__ float load_f(const __nv_bfloat16* p) {
  return __bfloat162float(*p);
}
__device__ __forceinline__ float load_f(const float* p) { return *p; }
__device__ __forceinline__ float load_f(const __half* p) {
  return __half2float(*p);
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, float v) {
  *p = __float2bfloat16_rn(v);
}
__device__ __forceinline__ void store16(__half* p, float v) {
  *p = __float2half_rn(v);
}

}  // namespace gemm_f32_impl
