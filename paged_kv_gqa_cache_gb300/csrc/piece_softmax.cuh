#pragma once
// The reference that a row's probabilities are taken against where P enters P V
// in two terms on the tcgen05 tiles (decode_shared.cu, attn_tree.cu), for sm_103a:
// P = 2^(s - m_ref), s the score in the log2 domain.
//
// A row's reference m_ref is kBelow under a maximum, and
// O is rescaled once a maximum is more than kTop above it.  bf16 has fp32's range:
// 0 and kRescale.  fp16 has 2^-25 to 65504, all of it used so that small weights
// are held nearly as in the split workers (decode_mma.cuh): P is 2^13 or more at the
// row's largest (a weight is off by 2^-38 of that one at most) and under 2^16.  The 2.9
// between the two decide how often O is rescaled (shared prefixes, 192 sequences in
// three groups, fp16: 108.7 us; with 14 and 15 in their place 118, 13 and 15 115.5, 12
// and 15 108; bf16 100.3).
#include "prefill_kernel.cuh"

namespace pa {
namespace {

template <typename T>
constexpr float kBelow = std::is_same<T, __half>::value ? 13.f : 0.f;
template <typename T>
constexpr float kTop = std::is_same<T, __half>::value ? 15.9f : kRescale;
template <typename T>
constexpr float kTopSum = std::is_same<T, __half>::value ? 61147.f : kRescaleSum;  // 2^kTop: a half-row sum bound
// The reference for a maximum mc, and what a maximum mc may reach above the
// reference: kBelow under it and kTop, while such sums are good to 2^-4; past that
// mc itself and nothing, since fp16 has no room for their roundings (weights under
// 2^-25 of the largest are then lost in fp16).
template <typename T>
__device__ __forceinline__ float reference_of(float mc) {
  return kBelow<T> == 0.f || fabsf(mc) >= 1048576.f ? mc : mc - kBelow<T>;
}
template <typename T>
__device__ __forceinline__ float top_of(float mc) {
  return kBelow<T> != 0.f && fabsf(mc) >= 1048576.f ? 0.f : kTop<T>;
}

}  // namespace
}  // namespace pa
