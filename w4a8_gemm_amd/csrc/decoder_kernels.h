// Launch interface of the decoder-layer operators: the int8 producers of the
// linear layers' inputs (norm, SwiGLU), and the paged int8 KV cache with its
// append and its attention.  The C ABI layer is decoder_api.cpp.
#pragma once
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "../../include/w4a8.h"

namespace w4a8 {

struct NormParams {
  const uint16_t* x;
  int ldx;
  const uint16_t* residual;   // may be null: h = x
  int ldr;
  const uint16_t* weight;
  float eps;
  int m, k;
  uint16_t* h;                // may be null without a residual
  int ldh;
  int8_t* a8;
  int lda8;
  uint16_t* s_a;
};

struct SwigluParams {
  const uint16_t* gate;
  int ldg;
  const uint16_t* up;
  int ldu;
  int m, k;
  int8_t* a8;
  int lda8;
  uint16_t* s_a;
};

hipError_t launch_rms_norm_quant(const NormParams& p, hipStream_t stream);
hipError_t launch_silu_mul_quant(const SwigluParams& p, hipStream_t stream);

// Turns a HIP status into the C ABI's and keeps it for
// w4a8_last_device_error (api.cpp).
w4a8_status device_status(hipError_t e);

}  // namespace w4a8
