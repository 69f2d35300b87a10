// C ABI entry points of the decoder-layer operators: argument validation
// (host only, before any HIP call) and launch plans.
#include <hip/hip_runtime_api.h>

#include <cmath>
#include <cstdint>

#include "../../include/w4a8.h"
#include "decoder_kernels.h"

using namespace w4a8;

extern "C" w4a8_status w4a8_rms_norm_quant(const uint16_t* x_dev, int ldx,
                                           const uint16_t* residual_dev, int ldr,
                                           const uint16_t* weight_dev, float eps, int m, int k,
                                           uint16_t* h_dev, int ldh, int8_t* a8_dev, int lda8,
                                           uint16_t* s_a_dev, void* stream) {
  if (m < 0 || m > W4A8_M_MAX || k <= 0 || k > W4A8_ACT_K_MAX || ldx < k || lda8 < k)
    return W4A8_ERR_INVALID_ARGUMENT;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return W4A8_ERR_INVALID_ARGUMENT;
  if (residual_dev && ldr < k) return W4A8_ERR_INVALID_ARGUMENT;
  if (h_dev && ldh < k) return W4A8_ERR_INVALID_ARGUMENT;
  if (m == 0) return W4A8_OK;
  if (!x_dev || !weight_dev || !a8_dev || !s_a_dev) return W4A8_ERR_INVALID_ARGUMENT;
  if (residual_dev && !h_dev) return W4A8_ERR_INVALID_ARGUMENT;
  NormParams p;
  p.x = x_dev;
  p.ldx = ldx;
  p.residual = residual_dev;
  p.ldr = ldr;
  p.weight = weight_dev;
  p.eps = eps;
  p.m = m;
  p.k = k;
  p.h = h_dev;
  p.ldh = ldh;
  p.a8 = a8_dev;
  p.lda8 = lda8;
  p.s_a = s_a_dev;
  return device_status(launch_rms_norm_quant(p, static_cast<hipStream_t>(stream)));
}

extern "C" w4a8_status w4a8_silu_mul_quant(const uint16_t* gate_dev, int ldg,
                                           const uint16_t* up_dev, int ldu, int m, int k,
                                           int8_t* a8_dev, int lda8, uint16_t* s_a_dev,
                                           void* stream) {
  if (m < 0 || m > W4A8_M_MAX || k <= 0 || k > W4A8_ACT_K_MAX || ldg < k || ldu < k || lda8 < k)
    return W4A8_ERR_INVALID_ARGUMENT;
  if (m == 0) return W4A8_OK;
  if (!gate_dev || !up_dev || !a8_dev || !s_a_dev) return W4A8_ERR_INVALID_ARGUMENT;
  SwigluParams p;
  p.gate = gate_dev;
  p.ldg = ldg;
  p.up = up_dev;
  p.ldu = ldu;
  p.m = m;
  p.k = k;
  p.a8 = a8_dev;
  p.lda8 = lda8;
  p.s_a = s_a_dev;
  return device_status(launch_silu_mul_quant(p, static_cast<hipStream_t>(stream)));
}
