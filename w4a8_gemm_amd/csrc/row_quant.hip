// Row operators that end in the per-token int8 quantizer (gfx950): the
// root-mean-square norm with the residual's addition, and silu(gate) * up.
// Both feed w4a8_gemm, so the fp16 row between them and the quantizer is
// never written.
//
// One workgroup per row.  A row's scale needs its largest |y|, and the
// norm's y needs the row's sum of squares.  Both come out of one reduction:
//   y = rstd * (h * w), and rounding rstd * t is monotone in |t|, so
//   max|y| = rstd * max|h * w| exactly as the codes see it.
//
// Bound by memory: rows stay in registers, so every byte moves once.  Over
// buffers that are not in the last-level cache, norm of 4096 x 8192 with residual
// (235 MB) takes 47 us = 5.0 TB/s, SwiGLU of 2048 x 24576 (252 MB) 51 us = 5.0
// TB/s; a large copy reaches 5.1 to 5.2.  On the same outputs again and again,
// partly cached, 41 and 47.  8 rows of 4096: 3.7 us, latency: the launch (1.5),
// one load from memory, the reduction through LDS, the codes' store.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "decoder_kernels.h"
#include "quant_common.h"

namespace w4a8 {
namespace {

using namespace dev;

// Rows of the norm from which up to 4 chunks a thread beat one (512 x 8192: 8.9
// us against 9.5, 4096 x 8192: 41 against 49; 256 x 8192: 5.6 against 5.5).
// Few rows leave compute units idle, and a row's time is its loads' latency;
// many rows share the units, and fewer waves a row spend less on the
// reduction.  SwiGLU, with an exponential and a reciprocal a value, takes one
// chunk a thread for any number of rows (2048 x 14336: 27 us against 30).
constexpr int kManyRows = 512;
constexpr int kThreads = 256;      // of the kernels for long or unaligned rows

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

// Largest |y| (as abs_bits) and the sum over a workgroup of T threads, in
// every thread; always added in the same order.
template <int T>
__device__ __forceinline__ void reduce(float& sum, uint32_t& mx) {
  __shared__ float sums[T / 64];
  __shared__ uint32_t maxs[T / 64];
  sum = wave_sum(sum);
  mx = wave_max_u32(mx);
  if ((threadIdx.x & 63) == 0) {
    sums[threadIdx.x >> 6] = sum;
    maxs[threadIdx.x >> 6] = mx;
  }
  __syncthreads();
  sum = 0.0f;
  mx = 0;
#pragma unroll
  for (int i = 0; i < T / 64; ++i) {
    sum += sums[i];
    mx = max(mx, maxs[i]);
  }
}

// eight codes under the multiplier r, one 8-byte store
__device__ __forceinline__ void store_codes(int8_t* dst, const float (&y)[8], float r) {
  uint32_t b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) b[j] = code_byte(y[j], r);
  uint2 o;
  o.x = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u) | __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
  o.y = __builtin_amdgcn_perm(b[5], b[4], 0x0c0c0400u) | __builtin_amdgcn_perm(b[7], b[6], 0x04000c0cu);
  *reinterpret_cast<uint2*>(dst) = o;
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  uint16_t v[8];
  __builtin_memcpy(v, &u, 16);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = h2f(v[j]);
}

// Rows that T threads hold in CH chunks of 8 values each: read once, all
// loads in flight together.
template <int T, int CH>
__global__ __launch_bounds__(T) void rms_norm_quant_held_kernel(NormParams p) {
  const int row = blockIdx.x, tid = threadIdx.x;
  const uint16_t* x = p.x + size_t(row) * size_t(p.ldx);
  uint4 v[CH], w[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (c * T + tid) * 8;
    v[c] = i < p.k ? *reinterpret_cast<const uint4*>(x + i) : uint4{0, 0, 0, 0};
  }
  if (p.residual) {
    const uint16_t* res = p.residual + size_t(row) * size_t(p.ldr);
    uint4 u[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * T + tid) * 8;
      u[c] = i < p.k ? *reinterpret_cast<const uint4*>(res + i) : uint4{0, 0, 0, 0};
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float a[8], b[8];
      unpack8(v[c], a);
      unpack8(u[c], b);
      uint16_t s[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = f2h_bits(a[j] + b[j]);
      __builtin_memcpy(&v[c], s, 16);
    }
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (c * T + tid) * 8;
    w[c] = i < p.k ? *reinterpret_cast<const uint4*>(p.weight + i) : uint4{0, 0, 0, 0};
  }
  if (p.h) {
    uint16_t* h = p.h + size_t(row) * size_t(p.ldh);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * T + tid) * 8;
      if (i < p.k) *reinterpret_cast<uint4*>(h + i) = v[c];
    }
  }
  float sum = 0.0f;
  uint32_t mx = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    float f[8], g[8];
    unpack8(v[c], f);
    unpack8(w[c], g);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sum = __builtin_fmaf(f[j], f[j], sum);
      mx = max(mx, abs_bits(f[j] * g[j]));
    }
  }
  reduce<T>(sum, mx);
  const float rstd = 1.0f / __builtin_sqrtf(sum / float(p.k) + p.eps);
  const uint16_t sb = scale_bits_of(rstd * __builtin_bit_cast(float, mx));
  if (tid == 0) p.s_a[row] = sb;
  const float r = act_recip(sb);
  int8_t* a8 = p.a8 + size_t(row) * size_t(p.lda8);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (c * T + tid) * 8;
    if (i >= p.k) continue;
    float f[8], g[8], y[8];
    unpack8(v[c], f);
    unpack8(w[c], g);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = rstd * (f[j] * g[j]);
    store_codes(a8 + i, y, r);
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
  reduce<kThreads>(sum, mx);
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
  float unused = 0.0f;
  reduce<kThreads>(unused, mx);
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

template <int T, int CH>
__global__ __launch_bounds__(T) void silu_mul_quant_held_kernel(SwigluParams p) {
  const int row = blockIdx.x, tid = threadIdx.x;
  const uint16_t* gate = p.gate + size_t(row) * size_t(p.ldg);
  const uint16_t* up = p.up + size_t(row) * size_t(p.ldu);
  uint4 g[CH], u[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (c * T + tid) * 8;
    g[c] = i < p.k ? *reinterpret_cast<const uint4*>(gate + i) : uint4{0, 0, 0, 0};
    u[c] = i < p.k ? *reinterpret_cast<const uint4*>(up + i) : uint4{0, 0, 0, 0};
  }
  float y[CH][8];
  uint32_t mx = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    uint16_t a[8], b[8];
    __builtin_memcpy(a, &g[c], 16);
    __builtin_memcpy(b, &u[c], 16);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      y[c][j] = swiglu(a[j], b[j]);
      mx = max(mx, abs_bits(y[c][j]));
    }
  }
  float unused = 0.0f;
  reduce<T>(unused, mx);
  const uint16_t sb = scale_bits_of(__builtin_bit_cast(float, mx));
  if (tid == 0) p.s_a[row] = sb;
  const float r = act_recip(sb);
  int8_t* a8 = p.a8 + size_t(row) * size_t(p.lda8);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (c * T + tid) * 8;
    if (i < p.k) store_codes(a8 + i, y[c], r);
  }
}

// Threads and chunks of a held row, with up to `most` chunks a thread before
// the threads are doubled (1024 threads take up to 4 in any case).  With many
// rows a few waves a row are enough and spend less on the reduction; with few,
// every thread takes one chunk if the row allows it, so that the loads of a
// row are all out at once.
struct Held {
  int threads, chunks;      // threads 0: the row is too long
};
Held held_plan(int m, int k, int most) {
  const int n = (k + 7) / 8;
  int t = 256;
  while (t < 1024 && n > most * t) t *= 2;
  // a launch holds fewer than 2^32 threads
  if (n > 4 * t || long(m) * t >= 1l << 32) return {0, 0};
  return {t, (n + t - 1) / t};
}

const void* norm_held(const Held& h) {
  if (h.threads == 256)
    return h.chunks == 1   ? reinterpret_cast<const void*>(&rms_norm_quant_held_kernel<256, 1>)
           : h.chunks == 2 ? reinterpret_cast<const void*>(&rms_norm_quant_held_kernel<256, 2>)
                           : reinterpret_cast<const void*>(&rms_norm_quant_held_kernel<256, 4>);
  if (h.threads == 512)
    return h.chunks == 1   ? reinterpret_cast<const void*>(&rms_norm_quant_held_kernel<512, 1>)
           : h.chunks <= 3 ? reinterpret_cast<const void*>(&rms_norm_quant_held_kernel<512, 3>)
                           : reinterpret_cast<const void*>(&rms_norm_quant_held_kernel<512, 4>);
  return h.chunks == 1   ? reinterpret_cast<const void*>(&rms_norm_quant_held_kernel<1024, 1>)
         : h.chunks == 2 ? reinterpret_cast<const void*>(&rms_norm_quant_held_kernel<1024, 2>)
         : h.chunks == 3 ? reinterpret_cast<const void*>(&rms_norm_quant_held_kernel<1024, 3>)
                         : reinterpret_cast<const void*>(&rms_norm_quant_held_kernel<1024, 4>);
}

const void* silu_mul_held(const Held& h) {
  if (h.threads == 256) return reinterpret_cast<const void*>(&silu_mul_quant_held_kernel<256, 1>);
  if (h.threads == 512) return reinterpret_cast<const void*>(&silu_mul_quant_held_kernel<512, 1>);
  return h.chunks == 1   ? reinterpret_cast<const void*>(&silu_mul_quant_held_kernel<1024, 1>)
         : h.chunks == 2 ? reinterpret_cast<const void*>(&silu_mul_quant_held_kernel<1024, 2>)
         : h.chunks == 3 ? reinterpret_cast<const void*>(&silu_mul_quant_held_kernel<1024, 3>)
                         : reinterpret_cast<const void*>(&silu_mul_quant_held_kernel<1024, 4>);
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
  const Held held = held_plan(p.m, p.k, p.m >= kManyRows ? 4 : 1);
  if (vec && held.threads)
    return hipLaunchKernel(norm_held(held), dim3(p.m), dim3(held.threads), args, 0, stream);
  const void* fn = vec ? reinterpret_cast<const void*>(&rms_norm_quant_kernel<true>)
                       : reinterpret_cast<const void*>(&rms_norm_quant_kernel<false>);
  return hipLaunchKernel(fn, dim3(p.m), dim3(kThreads), args, 0, stream);
}

hipError_t launch_silu_mul_quant(const SwigluParams& p, hipStream_t stream) {
  const bool vec = p.k % 8 == 0 && rows16(p.gate, p.ldg) && rows16(p.up, p.ldu) &&
                   rows8(p.a8, p.lda8);
  SwigluParams q = p;
  void* args[] = {&q};
  const Held held = held_plan(p.m, p.k, 1);
  if (vec && held.threads)
    return hipLaunchKernel(silu_mul_held(held), dim3(p.m), dim3(held.threads), args, 0, stream);
  const void* fn = vec ? reinterpret_cast<const void*>(&silu_mul_quant_kernel<true>)
                       : reinterpret_cast<const void*>(&silu_mul_quant_kernel<false>);
  return hipLaunchKernel(fn, dim3(p.m), dim3(kThreads), args, 0, stream);
}

}  // namespace w4a8
