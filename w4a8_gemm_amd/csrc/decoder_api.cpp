// C ABI entry points of the decoder-layer operators: argument validation
// (host only, before any HIP call) and launch plans.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/w4a8.h"
#include "decoder_checks.h"
#include "decoder_kernels.h"

using namespace w4a8;

namespace {

// What the attention launches for a batch: the kernel of 16-row tiles
// (waves == 0) or the one of 32 rows a wave, and the split of the keys.
struct AttnPlan {
  int waves;
  int splits, chunk;
  long wgs;
  size_t ml_bytes, workspace;
};

constexpr long kComputeUnits = 256;
constexpr int kMaxSplits = 256;
constexpr long kFewPartials = 1500000;

AttnPlan plan_attn(const KvArgs& kv, int q_heads, int max_q, int max_len) {
  AttnPlan pl;
  const int group = q_heads / kv.kv_heads;
  const long rows = long(kv.cu_q ? max_q : 1) * group;
  pl.waves = 0;
  if (rows > kAttnRows) {
    // 256 rows a workgroup (8 waves) where that fills the device, else 128
    const bool wide = kv.dim > 64 && kv.dim <= 128;
    pl.waves = wide && attn_tiles(kv, group, 256) * kv.kv_heads >= 3 * kComputeUnits ? 8 : 4;
  }
  const long units = attn_tiles(kv, group, pl.waves ? 32 * pl.waves : kAttnRows) * kv.kv_heads;
  // Keys per split: so many that about `target` workgroups of equal work run,
  // at least `least`; none for more rows than one launch joins.
  //   16-row tiles: 24 workgroups a compute unit even out ragged lengths
  //   (64 x up to 8192 keys: 6 a unit 142 us, 12 137, 24 131).
  //   Tiles of 128 or more rows: where the partial results, 4 bytes a value
  //   each way, are few, 3 a unit, unless the tiles make 2 a unit by themselves;
  //   where they are many, 2, and only if the tiles make less than one.  As many
  //   and as few, us: 16 x 8 tokens over 4000 keys (0.3 M values) 81 and 56,
  //   16 x 16 over 2048 (0.5 M) 59 and 40, 256 over 8000 (1.0 M) 83 and 72, 366
  //   over 8000 (1.5 M) 119 and 109, 3 x 700 over 1400 with heads of 64 (1.5 M)
  //   52 and 42; 440 over 8000 (1.8 M) 102 and 126, 512 over 8000 (2.1 M) 120 and
  //   134, 2000 over themselves (8 M) 71 and 123.  16 x 64 over 2048 (2.7 M) would
  //   gain from few, 77 and 73; most others between are equal.
  const long rows_all = long(kv.total_q) * q_heads;
  const bool few = rows_all * kv.dim <= kFewPartials;
  const long target = (!pl.waves ? 24 : few ? 3 : 2) * kComputeUnits;
  const double keys = double(units) * max_len;
  const long least = pl.waves ? 512 : keys >= 512.0 * 256 ? 256 : 128;
  double want = std::max(keys / double(target), double(max_len) / kMaxSplits);
  if (pl.waves && units >= (few ? 2 : 1) * kComputeUnits) want = max_len;
  if (rows_all > kMaxWgs256) want = max_len;
  const long chunk = std::max(1l, (long(want) + least) / least) * least;
  const long splits = std::max(1l, (max_len + chunk - 1) / chunk);
  pl.splits = int(splits);
  pl.chunk = int(std::min(chunk, 1l << 30));
  pl.wgs = units * splits;
  const size_t parts = splits > 1 ? size_t(rows_all) * size_t(splits) : 0;
  pl.ml_bytes = (parts * 8 + 255) / 256 * 256;
  pl.workspace = parts > 0 ? pl.ml_bytes + parts * size_t(kv.dim) * 4 : 0;
  return pl;
}

}  // namespace

extern "C" w4a8_status w4a8_rope_append_at(const uint16_t* q_dev, int ldq, const uint16_t* k_dev,
                                           int ldk, const uint16_t* v_dev, int ldv, int q_heads,
                                           const float* cos_sin_dev, int rotary_dim, int max_pos,
                                           int interleaved, const int32_t* positions_dev,
                                           const w4a8_kv_view* view, uint16_t* q_out_dev, int ldqo,
                                           void* stream) {
  AppendParams p;
  w4a8_status st = check_view(view, &p.kv);
  if (st != W4A8_OK) return st;
  if (rotary_dim < 0 || rotary_dim > view->head_dim || (rotary_dim > 0 && max_pos < 1))
    return W4A8_ERR_INVALID_ARGUMENT;
  if (rotary_dim % 16) return W4A8_ERR_UNSUPPORTED;
  if (q_heads < 1) return W4A8_ERR_INVALID_ARGUMENT;
  if (q_heads > W4A8_HEADS_MAX) return W4A8_ERR_UNSUPPORTED;
  if (view->batch == 0 || view->total_q == 0) return W4A8_OK;
  if (append_block_wgs(p.kv) + append_query_wgs(p.kv, q_heads) > kMaxWgs256)
    return W4A8_ERR_UNSUPPORTED;
  const long q_cols = long(q_heads) * p.kv.dim, kv_cols = long(p.kv.kv_heads) * p.kv.dim;
  if (!rows_ok(q_dev, ldq, q_cols) || !rows_ok(k_dev, ldk, kv_cols) ||
      !rows_ok(v_dev, ldv, kv_cols) || !rows_ok(q_out_dev, ldqo, q_cols))
    return W4A8_ERR_INVALID_ARGUMENT;
  if (rotary_dim > 0 && (!cos_sin_dev || !aligned16(cos_sin_dev))) return W4A8_ERR_INVALID_ARGUMENT;
  p.q = q_dev;
  p.k = k_dev;
  p.v = v_dev;
  p.q_out = q_out_dev;
  p.ldq = ldq;
  p.ldk = ldk;
  p.ldv = ldv;
  p.ldqo = ldqo;
  p.q_heads = q_heads;
  p.cos_sin = cos_sin_dev;
  p.rotary = rotary_dim;
  p.max_pos = max_pos;
  p.interleaved = interleaved;
  p.positions = positions_dev;
  return device_status(launch_rope_append(p, static_cast<hipStream_t>(stream)));
}

extern "C" w4a8_status w4a8_rope_append(const uint16_t* q_dev, int ldq, const uint16_t* k_dev,
                                        int ldk, const uint16_t* v_dev, int ldv, int q_heads,
                                        const float* cos_sin_dev, int rotary_dim, int max_pos,
                                        int interleaved, const w4a8_kv_view* view,
                                        uint16_t* q_out_dev, int ldqo, void* stream) {
  return w4a8_rope_append_at(q_dev, ldq, k_dev, ldk, v_dev, ldv, q_heads, cos_sin_dev, rotary_dim,
                             max_pos, interleaved, nullptr, view, q_out_dev, ldqo, stream);
}

extern "C" size_t w4a8_paged_attention_workspace_size(const w4a8_kv_view* view, int q_heads,
                                                      int max_q, int max_len) {
  KvArgs kv;
  if (check_view(view, &kv) != W4A8_OK || view->batch == 0 || view->total_q == 0) return 0;
  if (check_heads(kv, q_heads) != W4A8_OK || max_q < 0 || max_len < 0) return 0;
  return plan_attn(kv, q_heads, max_q, max_len).workspace;
}

extern "C" w4a8_status w4a8_paged_attention(const uint16_t* q_dev, int ldq, int q_heads,
                                            const w4a8_kv_view* view, int max_q, int max_len,
                                            float scale, int window, uint16_t* out_dev, int ldo,
                                            void* workspace_dev, size_t workspace_bytes,
                                            void* stream) {
  AttnParams p;
  w4a8_status st = check_view(view, &p.kv);
  if (st != W4A8_OK) return st;
  if (max_q < 0 || max_len < 0 || window < 0 || !std::isfinite(scale)) return W4A8_ERR_INVALID_ARGUMENT;
  if (view->batch == 0 || view->total_q == 0) return W4A8_OK;
  st = check_heads(p.kv, q_heads);
  if (st != W4A8_OK) return st;
  const long cols = long(q_heads) * p.kv.dim;
  if (!rows_ok(q_dev, ldq, cols) || !rows_ok(out_dev, ldo, cols)) return W4A8_ERR_INVALID_ARGUMENT;
  const AttnPlan pl = plan_attn(p.kv, q_heads, max_q, max_len);
  if (pl.wgs * (pl.waves == 8 ? 2 : 1) > kMaxWgs256) return W4A8_ERR_UNSUPPORTED;
  if (pl.workspace > 0) {
    if (workspace_bytes < pl.workspace) return W4A8_ERR_BUFFER_TOO_SMALL;
    if (!workspace_dev || !aligned16(workspace_dev)) return W4A8_ERR_INVALID_ARGUMENT;
  }
  p.q = q_dev;
  p.out = out_dev;
  p.ldq = ldq;
  p.ldo = ldo;
  p.q_heads = q_heads;
  p.group = q_heads / p.kv.kv_heads;
  p.scale_log2e = scale * 1.44269504f;
  p.window = window;
  p.splits = pl.splits;
  p.chunk = pl.chunk;
  p.part_ml = static_cast<float2*>(workspace_dev);
  p.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace_dev) + (pl.workspace ? pl.ml_bytes : 0));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  st = device_status(pl.waves ? launch_paged_attn_tile(p, pl.waves, s) : launch_paged_attn(p, s));
  if (st != W4A8_OK || pl.splits == 1) return st;
  return device_status(launch_attn_join(p, s));
}

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
