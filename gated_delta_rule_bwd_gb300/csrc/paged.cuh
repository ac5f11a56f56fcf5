// Pages of keys and values: where a row's slots lie, and 4-bit storage.
//
// 4-bit storage of a row of D values (one head of one token; D a multiple of
// 32): D / 2 bytes of codes, byte i the values 2 i (low four bits) and 2 i + 1,
// and a step per 32 values.
//   step = amax / 7 (the fp32 product with 1 / 7) rounded to 5 significant bits (half
//   up), held as bf16,
//   code = rint(x / step) in [-7, 7], held as code + 8;
// steps of 0 have codes of 0, and a NaN or infinity among the 32 makes the step
// NaN.  A code has 3 significant bits and a step 5, so that what a code stands
// for, code step, is a bf16 value without further rounding: kernels multiply
// exactly the values that are read back.  The step's own rounding moves it by at
// most 2^-5 of itself, and a largest value that then lies past 7 steps is still
// within half a step of code 7.
#pragma once

#include "attn_tc.cuh"

namespace gdn {
namespace paged {

constexpr int kStepGroup = 32;

__device__ __forceinline__ int sequence_of(const int* cu, int nseq, int tok) {
  int lo = 0, hi = nseq - 1;  // the last s with cu[s] <= tok
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (cu[mid] <= tok) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The step of values whose largest magnitude has these bits.
__device__ __forceinline__ float step_of(uint32_t amax) {
  if (amax >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  const float s = __fmul_rn(__uint_as_float(amax), 1.f / 7.f);
  return __uint_as_float((__float_as_uint(s) + 0x40000u) & 0xfff80000u);
}
__device__ __forceinline__ uint32_t code_of(float x, float step) {
  const float n = step > 0.f ? rintf(__fdiv_rn(x, step)) : 0.f;
  return (uint32_t)((int)fminf(fmaxf(n, -7.f), 7.f) + 8);
}
// Eight neighbouring values per lane, 32 in four neighbouring lanes: the lane's
// codes; `step` is the four lanes' own.  All lanes of the warp call.
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], float& step) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  step = step_of(m);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) w |= code_of(x[i], step) << (4 * i);
  return w;
}

// log2 of a page's tokens (a power of two)
inline int page_shift(int page) {
  int s = 0;
  while ((1 << s) < page) ++s;
  return s;
}

}  // namespace paged
}  // namespace gdn
