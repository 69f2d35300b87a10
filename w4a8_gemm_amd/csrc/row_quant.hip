// Row operators that end in the per-token int8 quantizer (gfx950): the
// root-mean-square norm with the residual's addition, and silu(gate) * up.
// Both feed w4a8_gemm, so the fp16 row between them and the quantizer is
// never written.
//
// One workgroup per row.  A row's scale needs its largest |y|, and the
// norm's y needs the row's sum of squares.  Both come out of one reduction:
//   y = rstd * (h * w), and rounding rstd * t is monotone in |t|, so
//   max|y| = rstd * max|h * w| exactly as the codes see it.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "decoder_kernels.h"
#include "quant_common.h"

namespace w4a8 {
namespace {

using namespace dev;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// |v| as an unsigned integer: ordered like the magnitude, with infinity above
// every finite value and NaN above infinity, so a maximum keeps both
__device__ __forceinline__ uint32_t abs_bits(float v) {
  return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
}

// low byte: the int8 code of y under the multiplier r (quant_byte, for fp32)
__device__ __forceinline__ uint32_t code_byte(float y, float r) {
  const float v = __builtin_amdgcn_fmed3f(y * r, -127.0f, 127.0f);
  return __builtin_bit_cast(uint32_t, v + 12582912.0f);
}

// s_a (fp16 bits) of a row whose largest |y| is amax
__device__ __forceinline__ uint16_t scale_bits_of(float amax) { return f2h_bits(amax / 127.0f); }

// Sum over the 64 lanes in every lane, always in the same order.
__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}

// 8 values of a row from i on: one 16-byte load, or value by value where the
// rows are not 16-byte aligned (the rest of a ragged end reads as 0)
template <bool VEC>
__device__ __forceinline__ void load8(const uint16_t* src, int i, int k, uint16_t (&v)[8]) {
  if (VEC) {
    const uint4 u = *reinterpret_cast<const uint4*>(src + i);
    __builtin_memcpy(v, &u, 16);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = i + j < k ? src[i + j] : uint16_t(0);
  }
}

template <bool VEC>
__device__ __forceinline__ void store8h(uint16_t* dst, int i, int k, const uint16_t (&v)[8]) {
  if (VEC) {
    uint4 u;
    __builtin_memcpy(&u, v, 16);
    *reinterpret_cast<uint4*>(dst + i) = u;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < k) dst[i + j] = v[j];
  }
}

template <bool VEC>
__device__ __forceinline__ void store8c(int8_t* dst, int i, int k, const float (&y)[8], float r) {
  uint32_t b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) b[j] = code_byte(y[j], r) & 0xFFu;
  if (VEC) {
    uint2 o;
    o.x = b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24;
    o.y = b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24;
    *reinterpret_cast<uint2*>(dst + i) = o;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < k) dst[i + j] = int8_t(uint8_t(b[j]));
  }
}

template <bool VEC>
__global__ __launch_bounds__(kThreads) void rms_norm_quant_kernel(NormParams p) {
  const int row = blockIdx.x, tid = threadIdx.x;
  const uint16_t* x = p.x + size_t(row) * size_t(p.ldx);
  const uint16_t* res = p.residual ? p.residual + size_t(row) * size_t(p.ldr) : nullptr;
  uint16_t* h = p.h ? p.h + size_t(row) * size_t(p.ldh) : nullptr;
  int8_t* a8 = p.a8 + size_t(row) * size_t(p.lda8);

  float sum = 0.0f;
  uint32_t mx = 0;
  for (int i = tid * 8; i < p.k; i += kThreads * 8) {
    uint16_t v[8], w[8];
    load8<VEC>(x, i, p.k, v);
    load8<VEC>(p.weight, i, p.k, w);
    if (res) {
      uint16_t u[8];
      load8<VEC>(res, i, p.k, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = f2h_bits(h2f(v[j]) + h2f(u[j]));
    }
    if (h) store8h<VEC>(h, i, p.k, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float f = h2f(v[j]);
      sum = __builtin_fmaf(f, f, sum);
      mx = max(mx, abs_bits(f * h2f(w[j])));
    }
  }
  __shared__ float wave_sums[kWaves];
  __shared__ uint32_t wave_maxs[kWaves];
  sum = wave_sum(sum);
  mx = wave_max_u32(mx);
  if ((tid & 63) == 0) {
    wave_sums[tid >> 6] = sum;
    wave_maxs[tid >> 6] = mx;
  }
  __syncthreads();
  sum = 0.0f;
  mx = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    sum += wave_sums[i];
    mx = max(mx, wave_maxs[i]);
  }
  const float rstd = 1.0f / __builtin_sqrtf(sum / float(p.k) + p.eps);
  const uint16_t sb = scale_bits_of(rstd * __builtin_bit_cast(float, mx));
  if (tid == 0) p.s_a[row] = sb;
  const float r = act_recip(sb);

  // the row again: what this thread stored to h, or x itself (then h == x)
  const uint16_t* again = h ? h : x;
  for (int i = tid * 8; i < p.k; i += kThreads * 8) {
    uint16_t v[8], w[8];
    load8<VEC>(again, i, p.k, v);
    load8<VEC>(p.weight, i, p.k, w);
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = rstd * (h2f(v[j]) * h2f(w[j]));
    store8c<VEC>(a8, i, p.k, y, r);
  }
}

// silu(g) * u in fp32, with the hardware's exp2 and reciprocal (about 1 ulp
// each; the result is rounded to 8 bits).  A large negative g makes exp2
// infinite and the quotient -0, a NaN stays one.
__device__ __forceinline__ float swiglu(uint16_t g16, uint16_t u16) {
  const float g = h2f(g16);
  const float e = __builtin_amdgcn_exp2f(g * -1.44269504f);
  return g * __builtin_amdgcn_rcpf(1.0f + e) * h2f(u16);
}

template <bool VEC>
__global__ __launch_bounds__(kThreads) void silu_mul_quant_kernel(SwigluParams p) {
  const int row = blockIdx.x, tid = threadIdx.x;
  const uint16_t* gate = p.gate + size_t(row) * size_t(p.ldg);
  const uint16_t* up = p.up + size_t(row) * size_t(p.ldu);
  int8_t* a8 = p.a8 + size_t(row) * size_t(p.lda8);

  uint32_t mx = 0;
  for (int i = tid * 8; i < p.k; i += kThreads * 8) {
    uint16_t g[8], u[8];
    load8<VEC>(gate, i, p.k, g);
    load8<VEC>(up, i, p.k, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) mx = max(mx, abs_bits(swiglu(g[j], u[j])));
  }
  __shared__ uint32_t wave_maxs[kWaves];
  mx = wave_max_u32(mx);
  if ((tid & 63) == 0) wave_maxs[tid >> 6] = mx;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWaves; ++i) mx = max(mx, wave_maxs[i]);
  const uint16_t sb = scale_bits_of(__builtin_bit_cast(float, mx));
  if (tid == 0) p.s_a[row] = sb;
  const float r = act_recip(sb);

  for (int i = tid * 8; i < p.k; i += kThreads * 8) {
    uint16_t g[8], u[8];
    load8<VEC>(gate, i, p.k, g);
    load8<VEC>(up, i, p.k, u);
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = swiglu(g[j], u[j]);
    store8c<VEC>(a8, i, p.k, y, r);
  }
}

bool rows16(const void* p, int ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0; }
bool rows8(const void* p, int ld) { return reinterpret_cast<uintptr_t>(p) % 8 == 0 && ld % 8 == 0; }

}  // namespace

hipError_t launch_rms_norm_quant(const NormParams& p, hipStream_t stream) {
  const bool vec = p.k % 8 == 0 && rows16(p.x, p.ldx) && rows16(p.weight, 0) &&
                   (!p.residual || rows16(p.residual, p.ldr)) && (!p.h || rows16(p.h, p.ldh)) &&
                   rows8(p.a8, p.lda8);
  NormParams q = p;
  void* args[] = {&q};
  const void* fn = vec ? reinterpret_cast<const void*>(&rms_norm_quant_kernel<true>)
                       : reinterpret_cast<const void*>(&rms_norm_quant_kernel<false>);
  return hipLaunchKernel(fn, dim3(p.m), dim3(kThreads), args, 0, stream);
}

hipError_t launch_silu_mul_quant(const SwigluParams& p, hipStream_t stream) {
  const bool vec = p.k % 8 == 0 && rows16(p.gate, p.ldg) && rows16(p.up, p.ldu) &&
                   rows8(p.a8, p.lda8);
  SwigluParams q = p;
  void* args[] = {&q};
  const void* fn = vec ? reinterpret_cast<const void*>(&silu_mul_quant_kernel<true>)
                       : reinterpret_cast<const void*>(&silu_mul_quant_kernel<false>);
  return hipLaunchKernel(fn, dim3(p.m), dim3(kThreads), args, 0, stream);
}

}  // namespace w4a8
