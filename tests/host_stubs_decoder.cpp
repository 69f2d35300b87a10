// Stand-ins for the device side of the decoder-layer operators, for a
// host-only build of decoder_api.cpp under AddressSanitizer and
// UndefinedBehaviorSanitizer.  A launch checks what the kernels assume of its
// parameters (grids and indices within their types) and reports no device.
#include <hip/hip_runtime_api.h>

#include <cstdlib>

#include "../w4a8_gemm_amd/csrc/decoder_kernels.h"

namespace w4a8 {

namespace {
void need(bool ok) {
  if (!ok) abort();
}
void check(const KvArgs& kv) {
  need(kv.data && kv.scale && kv.table && kv.lens && kv.num_pages > 0 && kv.kv_heads > 0);
  need(kv.dim >= 16 && kv.dim <= 256 && kv.dim % 16 == 0 && kv.page_shift >= 4 && kv.page_shift <= 10);
  need(kv.batch > 0 && kv.total_q > 0 && (kv.cu_q || kv.total_q == kv.batch));
  need((long(kv.max_pages) << kv.page_shift) < (1l << 31));
}
}  // namespace

w4a8_status device_status(hipError_t e) { return e == hipSuccess ? W4A8_OK : W4A8_ERR_DEVICE; }
hipError_t launch_rms_norm_quant(const NormParams& p, hipStream_t) {
  need(p.m > 0 && p.k > 0 && p.ldx >= p.k && p.lda8 >= p.k && (!p.residual || p.h));
  return hipErrorNoDevice;
}
hipError_t launch_silu_mul_quant(const SwigluParams& p, hipStream_t) {
  need(p.m > 0 && p.k > 0 && p.ldg >= p.k && p.ldu >= p.k && p.lda8 >= p.k);
  return hipErrorNoDevice;
}
hipError_t launch_rope_append(const AppendParams& p, hipStream_t) {
  check(p.kv);
  need(append_block_wgs(p.kv) + append_query_wgs(p.kv, p.q_heads) <= kMaxWgs256);
  need(append_slots(p.kv) * 2 * p.kv.kv_heads < (1l << 31) && p.rotary % 16 == 0);
  return hipErrorNoDevice;
}
namespace {
hipError_t attn(const AttnParams& p, int rows) {
  check(p.kv);
  need(p.splits >= 1 && p.splits <= 256 && p.chunk > 0 && p.chunk % 64 == 0);
  need(attn_tiles(p.kv, p.group, rows) * p.kv.kv_heads * p.splits <= kMaxWgs256);
  need(p.group * p.kv.kv_heads == p.q_heads && (p.splits == 1 || p.part_ml));
  return hipErrorNoDevice;
}
}  // namespace
hipError_t launch_paged_attn(const AttnParams& p, hipStream_t) { return attn(p, kAttnRows); }
hipError_t launch_paged_attn_tile(const AttnParams& p, int waves, hipStream_t) {
  need(waves == 4 || (waves == 8 && p.kv.dim > 64 && p.kv.dim <= 128));
  return attn(p, 32 * waves);
}
hipError_t launch_attn_join(const AttnParams&, hipStream_t) { return hipErrorNoDevice; }

}  // namespace w4a8
