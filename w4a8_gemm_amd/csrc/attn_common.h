// Device helpers of the attention kernels over the paged int8 cache (gfx950):
// int8 codes to fp16 matrix operands.
//
// Codes enter the fp16 matrix cores as exact integers: |code| <= 127 fits
// fp16's 11 bits.  Scales never touch a key or value.  A page's key scale
// multiplies its scores (in the fp32 factor that scales them anyway), and a
// page's value scale sv joins the softmax weight in the exponent:
//   sum_t p_t sv_t code_t  with  p_t sv_t = exp2(score_t + log2 sv_t - M),
// M the running maximum of score + log2 sv.  The weights' own sum divides
// sv out again, page by page, in fp32, from the weights before they are rounded
// to fp16: a page of small values has weights far below the others', whose
// few bits do for its values but not for its part of the sum.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "quant_common.h"

namespace w4a8 {
namespace attn {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// A finite "no key yet", below every score: exp2(-inf - kNone) is 0, not NaN.
static constexpr float kNone = -3.4028235e38f;
// Softmax weights are kept up to 2^kLift, so that weights down to 2^-(24 +
// kLift) of the largest still register in fp16; the sum carries the same
// factor and the quotient drops it.
static constexpr float kLift = 10.0f;
// Scores more than 2^kRoom above a row's maximum move it (fp16 ends at 2^16).
static constexpr float kRoom = 15.0f;

// A page's key scale.  An infinite one becomes NaN, and with it the scores of its
// keys: infinity times a negative sum would be the score of a masked key.
static __device__ __forceinline__ float key_scale(uint32_t bits) {
  const float s = dev::h2f(uint16_t(bits));
  return s + (s - s);
}

// Queries as they enter the product: an infinity becomes NaN, and with it every
// score of the row, where minus infinity would be the score of a masked key.
static __device__ __forceinline__ half8_t query8(half8_t q) { return q + (q - q); }

// A row's maximum, less the lift.  Scores from 2^27 on are 16 and more apart: the
// difference may round to one that leaves fp16's range, and goes without then.
static __device__ __forceinline__ float lifted(float mx) {
  const float m = mx - kLift;
  return mx - m > kRoom ? mx : m;
}

// codes as unsigned bytes (code + 128), four at a time
static __device__ __forceinline__ uint32_t biased(uint32_t w) { return w ^ 0x80808080u; }

// two biased bytes b0, b1, each the low byte of a 16-bit half, as
// fp16(code * 2^-9): a half whose bits are an integer u <= 255 is the
// subnormal u * 2^-24, so one packed fused multiply-add with 2^15 and
// -128 * 2^-9 gives (u - 128) * 2^-9 exactly.
static constexpr float kCodeScale = 512.0f;     // 2^9, to multiply results with
static __device__ __forceinline__ half2_t codes2(uint32_t halves) {
  const half2_t u = __builtin_bit_cast(half2_t, halves);
  const half2_t a = {(_Float16)32768.0f, (_Float16)32768.0f};
  const half2_t c = {(_Float16)-0.25f, (_Float16)-0.25f};
  return __builtin_elementwise_fma(u, a, c);
}

// 8 consecutive codes (two dwords, biased) as fp16 * 2^-9
static __device__ __forceinline__ half8_t codes8(uint32_t lo, uint32_t hi) {
  half8_t r;
  const half2_t a = codes2(__builtin_amdgcn_perm(0u, lo, 0x0c010c00u));
  const half2_t b = codes2(__builtin_amdgcn_perm(0u, lo, 0x0c030c02u));
  const half2_t c = codes2(__builtin_amdgcn_perm(0u, hi, 0x0c010c00u));
  const half2_t d = codes2(__builtin_amdgcn_perm(0u, hi, 0x0c030c02u));
  r[0] = a[0], r[1] = a[1], r[2] = b[0], r[3] = b[1];
  r[4] = c[0], r[5] = c[1], r[6] = d[0], r[7] = d[1];
  return r;
}

// byte `col` (0..3, a constant) of two dwords as two 16-bit halves: w0's first
static __device__ __forceinline__ uint32_t pair_bytes(uint32_t w0, uint32_t w1, int col) {
  return __builtin_amdgcn_perm(w1, w0, 0x0c040c00u + 0x00010001u * uint32_t(col));
}

static __device__ __forceinline__ f32x4 mfma16(half8_t a, half8_t b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

}  // namespace attn
}  // namespace w4a8
