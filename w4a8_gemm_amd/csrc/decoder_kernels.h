// Launch interface of the decoder-layer operators: the int8 producers of the
// linear layers' inputs (norm, SwiGLU), and the paged int8 KV cache with its
// append and its attention.  The C ABI layer is decoder_api.cpp.
#pragma once
#include <stdint.h>

#include <hip/hip_runtime_api.h>
#include <hip/hip_vector_types.h>

#include "../../include/w4a8.h"

namespace w4a8 {

// A launch holds fewer than 2^32 threads: workgroups of 256, checked by the
// C ABI layer before any HIP call.
constexpr long kMaxWgs256 = (1l << 24) - 1;

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

// The paged cache and the batch that one call reads or writes (the C ABI's
// w4a8_kv_view, validated), as the kernels take it.
struct KvArgs {
  int8_t* data;               // [num_pages][2][kv_heads][page][dim], pages page_stride apart
  uint16_t* scale;            // [num_pages][2][kv_heads], pages scale_stride apart
  long page_stride, scale_stride;
  int num_pages, kv_heads, dim;
  int page_shift;             // page size = 1 << page_shift
  const int32_t* table;
  int table_ld, max_pages;
  const int32_t* lens;
  const int32_t* cu_q;        // null: one new token per sequence
  int batch, total_q;
};

struct AppendParams {
  KvArgs kv;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* q_out;
  int ldq, ldk, ldv, ldqo;
  int q_heads;
  const float* cos_sin;       // [max_pos][rotary]: cosines, then sines
  int rotary, max_pos;
  int interleaved;
};

// Virtual page slots of an append: sequence b's written pages have the
// indices floor(cu_q[b] / page) + 2b ... (a sequence of n tokens touches at
// most floor(n / page) + 2 pages wherever it starts, so the ranges are
// disjoint); one slot per sequence where each brings one token.
inline long append_slots(const KvArgs& kv) {
  return kv.cu_q ? (long(kv.total_q) >> kv.page_shift) + 2l * kv.batch : long(kv.batch);
}
// One wave per block of the cache, and one head of a query per thread, where a
// block's new values are at most 128 items of 16 (two a lane): 64 x 16 tokens
// into pages of 16 7.5 us against 12.8 with a workgroup per block, 4 x 1500
// into pages of 16 22.3 against 27.9; beyond, a workgroup per block and 4
// heads a thread (pages of 32 22.3 against 23.5, of 64 22.8 against 27.1).
inline bool append_small(const KvArgs& kv) {
  const long each = (long(kv.total_q) + kv.batch - 1) / kv.batch;
  const long page = 1l << kv.page_shift;
  return (each < page ? each : page) * (kv.dim / 16) <= 128;
}
// workgroups of 256 threads: those that own blocks, then those of the queries
inline long append_block_wgs(const KvArgs& kv) {
  const long units = append_slots(kv) * 2 * kv.kv_heads;
  return append_small(kv) ? (units + 3) / 4 : units;
}
inline long append_query_wgs(const KvArgs& kv, int q_heads) {
  const int heads = append_small(kv) ? 1 : 4;
  return (long(kv.total_q) * (kv.dim / 16) * ((q_heads + heads - 1) / heads) + 255) / 256;
}
hipError_t launch_rope_append(const AppendParams& p, hipStream_t stream);

struct AttnParams {
  KvArgs kv;
  const uint16_t* q;
  uint16_t* out;
  int ldq, ldo;
  int q_heads, group;         // group = q_heads / kv_heads
  float scale_log2e;          // score scale * log2(e)
  int window;                 // 0: none
  int splits;                 // workgroups that split one row tile's keys,
  int chunk;                  // and the keys of each (a multiple of 64; the last takes the rest)
  float2* part_ml;            // splits > 1: maximum and sum of [token][query head][split],
  float* part_o;              // and its unnormalised values, [dim] each
};

// Row tiles of the attention: the rows of a sequence and kv head are its
// (token, query head of the group) pairs, tiled by `rows`; sequence b's
// tiles have the indices floor(cu_q[b] * group / rows) + b ...
inline long attn_tiles(const KvArgs& kv, int group, int rows) {
  return kv.cu_q ? long(kv.total_q) * group / rows + kv.batch
                 : long(kv.batch) * ((group + rows - 1) / rows);
}
constexpr int kAttnRows = 16;   // rows of a tile (paged_attn.hip)
hipError_t launch_paged_attn(const AttnParams& p, hipStream_t stream);
// 32 rows a wave, 4 waves, or 8 where 64 < dim <= 128 (paged_attn_tile.hip)
hipError_t launch_paged_attn_tile(const AttnParams& p, int waves, hipStream_t stream);
hipError_t launch_attn_join(const AttnParams& p, hipStream_t stream);

// Turns a HIP status into the C ABI's and keeps it for
// w4a8_last_device_error (api.cpp).
w4a8_status device_status(hipError_t e);

}  // namespace w4a8
