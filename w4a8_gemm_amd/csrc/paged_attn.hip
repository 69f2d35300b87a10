// Attention over the paged int8 cache (gfx950).
//
// A row is one (query token, query head); the rows of a sequence and kv head
// share keys and values and are tiled 16 at a time.  Four waves share a
// row tile, each taking every fourth step of 32 keys straight from memory
// into registers, and join through LDS; where there are few row tiles, the
// keys are split over workgroups as well and attn_join_kernel joins them.
//
// Both products run transposed on v_mfma_f32_16x16x32_f16:
//   S^T[key, row] = K Q^T      keys are rows of A, 16 per product
//   O^T[d, row]  += V^T P^T    values transposed on the way in
// so that a lane's accumulators all belong to one row (lane % 16).  Softmax
// statistics are then per lane, and P^T leaves the first product in the very
// registers the second one takes it from: quarter q of the wave holds keys
// 4q .. 4q + 3 of each 16-key half, and the second product's 8 k-slots of
// that quarter are those 4 + 4 keys.  A lane reads 8 keys x DP/16 value
// columns and picks one column's bytes for each product, so column d of V
// is result row (d / (DP/16), d % (DP/16)) and a lane ends with DP/16
// neighbouring values of one row.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn_common.h"
#include "decoder_kernels.h"
#include "kv_page.h"
#include "quant_common.h"

namespace w4a8 {
namespace {

using namespace attn;
using namespace dev;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = 32;      // keys a wave takes at once

// maximum over the four lanes of a row (lane, lane ^ 16, lane ^ 32, ...)
__device__ __forceinline__ float row_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float row_sum(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

// The keys of one 16-key half step: where they lie and their scales.
struct Half {
  const int8_t* k;    // 16 keys x dim codes
  const int8_t* v;
  float sk;           // key scale (with the score factor)
  float lv, rv;       // log2 and reciprocal of the value scale
  bool ok;            // the page exists
};

// Partial results of a split row: l, M and the unnormalised O, as
// part[(token * heads + head) * splits + split][dim + 2].

// DP: head dim rounded up to 64, 128 or 256.  PAD: dim < DP.
template <int DP, bool PAD>
__global__ __launch_bounds__(kThreads) void attn_split_kernel(AttnParams p) {
  constexpr int kQuarter = DP / 4;        // K bytes of a lane and key
  constexpr int kKStep = DP / 32;         // products of one 16-key score tile
  constexpr int kCols = DP / 16;          // V columns of a lane
  constexpr int kVDwords = DP / 64;       // dwords of those columns and one key
  const KvArgs& kv = p.kv;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, quarter = lane >> 4;

  const int split = blockIdx.x % p.splits;
  const int rest = blockIdx.x / p.splits;
  const int head = rest % kv.kv_heads;
  const int tile = rest / kv.kv_heads;
  int b, nth;
  if (kv.cu_q) {
    b = kv::owner(tile, kv.batch,
                  [&](int i) { return int(long(kv.cu_q[i]) * p.group / kAttnRows) + i; }, &nth);
  } else {
    const int per = (p.group + kAttnRows - 1) / kAttnRows;
    b = tile / per;
    nth = tile - b * per;
  }
  const kv::Seq s = kv::seq_of(kv, b);
  const int rows = (s.hi - s.lo) * p.group;
  if (nth < 0 || long(nth) * kAttnRows >= rows) return;   // the whole workgroup
  const int row = nth * kAttnRows + r16;
  const bool row_ok = row < rows;
  const int t = row / p.group;                       // new token of this lane's row
  const int q_head = head * p.group + row - t * p.group;
  const int pos = s.len - (s.hi - s.lo) + t;
  // keys this row sees: [see_lo, see_hi)
  const int see_hi = row_ok ? pos + 1 : 0;
  const int see_lo = p.window > 0 ? max(pos - p.window + 1, 0) : 0;
  // keys the tile sees
  const int t_first = nth * kAttnRows / p.group;
  const int t_last = (min(rows, (nth + 1) * kAttnRows) - 1) / p.group;
  const int pos_first = s.len - (s.hi - s.lo) + t_first;
  const int all_hi = max(s.len - (s.hi - s.lo) + t_last + 1, 0);
  const int all_lo = p.window > 0 ? max(pos_first - p.window + 1, 0) : 0;
  const int step0 = all_lo / kStep;
  const int steps = max((all_hi + kStep - 1) / kStep - step0, 0);
  const int first = step0 + int(long(steps) * split / p.splits);
  const int last = step0 + int(long(steps) * (split + 1) / p.splits);

  // Q^T fragments: lane's row, d = quarter * DP/4 + 8 s ..
  half8_t q[kKStep];
  {
    const uint16_t* src = p.q + long(s.lo + t) * p.ldq + long(q_head) * kv.dim;
#pragma unroll
    for (int i = 0; i < kKStep; ++i) {
      const int d = quarter * kQuarter + 8 * i;
      uint4 u = {0, 0, 0, 0};
      if (row_ok && (!PAD || d < kv.dim)) u = *reinterpret_cast<const uint4*>(src + d);
      q[i] = __builtin_bit_cast(half8_t, u);
    }
  }

  f32x4 o[kCols];
#pragma unroll
  for (int j = 0; j < kCols; ++j) o[j] = f32x4{0, 0, 0, 0};
  float m = kNone, l = 0.0f;

  const long head_bytes = long(kv.dim) << kv.page_shift;
  for (int st = first + wave; st < last; st += kWaves) {
    const int key0 = st * kStep;
    Half hf[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int key = key0 + 16 * u;
      const int page = key < all_hi ? kv::page_at(kv, b, key >> kv.page_shift) : -1;
      hf[u].ok = page >= 0;
      const int at = max(page, 0);
      const int slot = key & ((1 << kv.page_shift) - 1);
      const int8_t* base = kv.data + long(at) * kv.page_stride + head * head_bytes + long(slot) * kv.dim;
      hf[u].k = base;
      hf[u].v = base + kv.kv_heads * head_bytes;
      const uint16_t* sc = kv.scale + long(at) * kv.scale_stride + head;
      hf[u].sk = h2f(sc[0]) * p.scale_log2e * kCodeScale;
      // an all-zero page has scale 0: any positive value does, and the
      // smallest leaves the running maximum to the other pages
      const float sv = h2f(sc[kv.kv_heads]);
      const float sv1 = sv == 0.0f ? 0x1p-24f : sv;
      hf[u].lv = __builtin_amdgcn_logf(sv1);
      hf[u].rv = __builtin_amdgcn_rcpf(sv1);
    }
    // scores
    float x[8];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f32x4 acc = {0, 0, 0, 0};
      uint32_t w[DP / 16];
#pragma unroll
      for (int c = 0; c < DP / 64; ++c) {
        const int d = quarter * kQuarter + 16 * c;
        uint4 v = {0, 0, 0, 0};
        if (!PAD || d < kv.dim) v = *reinterpret_cast<const uint4*>(hf[u].k + r16 * kv.dim + d);
        w[4 * c] = v.x, w[4 * c + 1] = v.y, w[4 * c + 2] = v.z, w[4 * c + 3] = v.w;
      }
#pragma unroll
      for (int i = 0; i < kKStep; ++i)
        acc = mfma16(codes8(biased(w[2 * i]), biased(w[2 * i + 1])), q[i], acc);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = key0 + 16 * u + quarter * 4 + i;
        const bool seen = hf[u].ok && key >= see_lo && key < see_hi;
        x[4 * u + i] = seen ? __builtin_fmaf(acc[i], hf[u].sk, hf[u].lv) : -__builtin_inff();
      }
    }
    float mx = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) mx = fmaxf(mx, x[i]);
    const float m_new = fmaxf(m, row_max(mx) - kLift);
    const float alpha = __builtin_amdgcn_exp2f(m - m_new);
    m = m_new;
    half8_t pt;
    float sum[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float e = __builtin_amdgcn_exp2f(x[i] - m);
      sum[i >> 2] += e;
      pt[i] = static_cast<_Float16>(e);
    }
    l *= alpha;
    // a sum of 0 (nothing seen) stays 0 whatever the page's scale holds
#pragma unroll
    for (int u = 0; u < 2; ++u) l += sum[u] == 0.0f ? 0.0f : sum[u] * hf[u].rv;
#pragma unroll
    for (int j = 0; j < kCols; ++j) o[j] *= alpha;

    // values: 8 keys x kCols columns
    uint32_t vw[8][kVDwords];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int8_t* src = hf[i >> 2].v + (quarter * 4 + (i & 3)) * kv.dim + r16 * kCols;
#pragma unroll
      for (int c = 0; c < kVDwords; ++c) {
        uint32_t v = 0;
        if (!PAD || r16 * kCols < kv.dim) v = *reinterpret_cast<const uint32_t*>(src + 4 * c);
        vw[i][c] = biased(v);
      }
    }
#pragma unroll
    for (int c = 0; c < kVDwords; ++c) {
#define W4A8_COLUMN(B)                                                          \
  {                                                                             \
    half8_t a;                                                                  \
    _Pragma("unroll") for (int i = 0; i < 8; i += 2) {                          \
      const half2_t two = codes2(pair_bytes<B>(vw[i][c], vw[i + 1][c]));        \
      a[i] = two[0];                                                            \
      a[i + 1] = two[1];                                                        \
    }                                                                           \
    o[4 * c + B] = mfma16(a, pt, o[4 * c + B]);                                 \
  }
      W4A8_COLUMN(0)
      W4A8_COLUMN(1)
      W4A8_COLUMN(2)
      W4A8_COLUMN(3)
#undef W4A8_COLUMN
    }
  }
  l = row_sum(l);

  // O^T tile j: lane holds result rows 4 quarter + i, i.e. columns
  // (4 quarter + i) * kCols + j of its row.  Join the four waves: two LDS
  // arrays of statistics, then the sums themselves, 4 columns at a time.
  __shared__ float sh_m[kWaves][16], sh_l[kWaves][16];
  __shared__ f32x4 sh_o[kWaves][64][kCols + 1];
  if (quarter == 0) {
    sh_m[wave][r16] = m;
    sh_l[wave][r16] = l;
  }
#pragma unroll
  for (int j = 0; j < kCols; ++j) sh_o[wave][lane][j] = o[j];
  __syncthreads();
  float m_all = sh_m[0][r16];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) m_all = fmaxf(m_all, sh_m[w][r16]);
  float l_all = 0.0f, factor[kWaves];
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    factor[w] = __builtin_amdgcn_exp2f(sh_m[w][r16] - m_all);
    l_all += sh_l[w][r16] * factor[w];
  }
  if (!row_ok) return;
  const float norm = l_all > 0.0f || l_all != l_all ? kCodeScale / l_all : 0.0f;
  // wave w finishes result row i = w of each quarter: kCols columns
  const int i = wave;
  const int d0 = (4 * quarter + i) * kCols;
  if (PAD && d0 >= kv.dim) return;
  float out[kCols];
#pragma unroll
  for (int j = 0; j < kCols; ++j) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += sh_o[w][lane][j][i] * factor[w];
    out[j] = v;
  }
  if (p.splits == 1) {
    uint16_t* dst = p.out + long(s.lo + t) * p.ldo + long(q_head) * kv.dim + d0;
#pragma unroll
    for (int j = 0; j < kCols; ++j) dst[j] = f2h_bits(out[j] * norm);
  } else {
    float* dst = p.part + ((long(s.lo + t) * p.q_heads + q_head) * p.splits + split) * (kv.dim + 2);
    if (quarter == 0 && i == 0) {
      dst[0] = l_all;
      dst[1] = m_all;
    }
#pragma unroll
    for (int j = 0; j < kCols; ++j) dst[2 + d0 + j] = out[j];
  }
}

// One wave per row: the row's splits, in their order.
__global__ __launch_bounds__(256) void attn_join_kernel(AttnParams p) {
  const int dim = p.kv.dim;
  const long row = long(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (row >= long(p.kv.total_q) * p.q_heads) return;
  const float* src = p.part + row * p.splits * (dim + 2);
  float m = kNone;
  for (int s = 0; s < p.splits; ++s) m = fmaxf(m, src[long(s) * (dim + 2) + 1]);
  float l = 0.0f;
  for (int s = 0; s < p.splits; ++s)
    l += src[long(s) * (dim + 2)] * __builtin_amdgcn_exp2f(src[long(s) * (dim + 2) + 1] - m);
  const float norm = l > 0.0f || l != l ? kCodeScale / l : 0.0f;
  const long t = row / p.q_heads;
  uint16_t* dst = p.out + t * p.ldo + (row - t * p.q_heads) * dim;
  for (int d = lane; d < dim; d += 64) {
    float v = 0.0f;
    for (int s = 0; s < p.splits; ++s) {
      const float* part = src + long(s) * (dim + 2);
      v += part[2 + d] * __builtin_amdgcn_exp2f(part[1] - m);
    }
    dst[d] = f2h_bits(v * norm);
  }
}

}  // namespace

hipError_t launch_paged_attn(const AttnParams& p, hipStream_t stream) {
  AttnParams a = p;
  void* args[] = {&a};
  const long wgs = attn_tiles(p.kv, p.group, kAttnRows) * p.kv.kv_heads * p.splits;
  if (wgs > 2147483647l) return hipErrorInvalidValue;
  const int dim = p.kv.dim;
  const void* fn;
  if (dim == 64) fn = reinterpret_cast<const void*>(&attn_split_kernel<64, false>);
  else if (dim < 64) fn = reinterpret_cast<const void*>(&attn_split_kernel<64, true>);
  else if (dim == 128) fn = reinterpret_cast<const void*>(&attn_split_kernel<128, false>);
  else if (dim < 128) fn = reinterpret_cast<const void*>(&attn_split_kernel<128, true>);
  else if (dim == 256) fn = reinterpret_cast<const void*>(&attn_split_kernel<256, false>);
  else fn = reinterpret_cast<const void*>(&attn_split_kernel<256, true>);
  return hipLaunchKernel(fn, dim3(unsigned(wgs)), dim3(kThreads), args, 0, stream);
}

hipError_t launch_attn_join(const AttnParams& p, hipStream_t stream) {
  AttnParams a = p;
  void* args[] = {&a};
  const long rows = long(p.kv.total_q) * p.q_heads;
  return hipLaunchKernel(reinterpret_cast<const void*>(&attn_join_kernel),
                         dim3(unsigned((rows + 3) / 4)), dim3(256), args, 0, stream);
}

}  // namespace w4a8
