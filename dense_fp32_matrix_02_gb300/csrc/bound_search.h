// A search for a bound that at least k of some 32-bit keys reach, and not many
// more: the range of the keys in at most 256 steps, and the step with the k-th
// largest in 256 again while it holds many.  Host code too: the search is tested
// without a GPU.
//
// It ends whatever the keys are.  The range need not hold them (where the
// products gave up it comes from maxima that belong to no logits): a key above
// it counts as its last one, so that no step lies past the range's end, every
// range lies in the one before, and is at most 1/128 as wide.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define GEMM_F32_HD __host__ __device__ __forceinline__
#else
#define GEMM_F32_HD inline
#endif

namespace gemm_f32_impl {

constexpr int kBoundBins = 256;
constexpr int kBoundRounds = 4;  // 2^32 / 256^4

// The step of a key >= low.
GEMM_F32_HD uint32_t bound_bin(uint32_t key, uint32_t low, uint32_t high,
                               int shift) {
  return ((key < high ? key : high) - low) >> shift;
}

// count(low, high, shift, in_step): the step with the k-th largest key, by
// bound_bin of those >= low, and how many keys are in it.
template <typename Count>
GEMM_F32_HD uint32_t bound_search(uint32_t low, uint32_t high, int enough,
                                  Count count) {
  if (high < low) high = low;
  for (int round = 0; round < kBoundRounds; ++round) {
    int shift = 0, in_step = 0;
    while ((high - low) >> shift >= (uint32_t)kBoundBins) ++shift;
    low += (uint32_t)count(low, high, shift, in_step) << shift;
    const uint32_t end = low + ((1u << shift) - 1u);
    if (end < high) high = end;
    if (in_step <= enough || shift == 0) break;
  }
  return low;
}

}  // namespace gemm_f32_impl
