// Attention over the paged int8 cache (gfx950).
//
// A row is one (query token, query head); the rows of a sequence and kv head
// share keys and values and are tiled 16 at a time.  Four waves share a
// row tile, each taking every fourth step of 32 keys straight from memory
// into registers, and join through LDS; where there are few row tiles, the
// keys are split over workgroups as well, in chunks of the same number of
// keys for every sequence, and attn_join_kernel joins them.
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
//
// Bound by memory: every key and value byte is read once.  Measured, graph
// replays with the join: 64 sequences of up to 8192 keys (673 MB) 132 to 136 us =
// 5.0 TB/s, 16 x 64 heads x up to 4000 keys in pages of 16 (637 MB) 124 to 127 us
// = 5.1 TB/s, two of up to 131072 (366 MB) 81 to 84 us = 4.4 TB/s, where a large
// copy reaches 5.2 TB/s and a kernel that only reads 6 to 7; one of 2001 keys
// 9.4 us, two launches and their chains of loads.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn_common.h"
#include "decoder_kernels.h"
#include "kv_page.h"
#include "quant_common.h"
#include "tile_common.h"

namespace w4a8 {
namespace {

using namespace attn;
using namespace dev;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = 32;      // keys a wave takes at once
// Rows that get four waves each in the join: 64 rows of 30000 keys 22.0 us in all
// against 26.2 with one wave, 1024 rows of 1000 keys 15.7 each way, 2048 rows
// 20.1 against 18.7.
constexpr long kJoinFewRows = 1024;

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// maximum over the four lanes of a row (lane, lane ^ 16, lane ^ 32, ...)
__device__ __forceinline__ float row_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float row_sum(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

// The 32 keys of a step on their way to the matrix cores: codes as loaded,
// and the scales (raw fp16) of the two 16-key halves.
template <int DP>
struct Step {
  u32x4 k[2][DP / 64];
  uint32_t v[8][DP / 64];
  uint32_t sk[2], sv[2];
  bool ok[2];                   // the half's page exists
};

// DP: head dim rounded up to 64, 128 or 256.  PAD: dim < DP.
template <int DP, bool PAD>
__global__ __launch_bounds__(kThreads, DP == 256 ? 2 : 4) void attn_split_kernel(AttnParams p) {
  constexpr int kQuarter = DP / 4;        // K bytes of a lane and key
  constexpr int kKStep = DP / 32;         // products of one 16-key score tile
  constexpr int kCols = DP / 16;          // V columns of a lane
  constexpr int kVDwords = DP / 64;       // dwords of those columns and one key
  const KvArgs& kv = p.kv;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, quarter = lane >> 4;

  // Splits fastest, turned from row tile to row tile: workgroups go round the
  // 8 dies in turn, and without the turn a power of two of splits would give
  // some dies only the splits that lie beyond short sequences (16 x 64
  // heads x 4000 keys in 2 splits: 167 us, turned 125).
  const int rest = blockIdx.x / p.splits;
  const int split = (blockIdx.x % p.splits + (rest >> 2)) % p.splits;
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
  const int start = s.len - (s.hi - s.lo);           // position of the first new token
  const int row = nth * kAttnRows + r16;
  const bool row_ok = row < rows;
  const int t = row / p.group;                       // new token of this lane's row
  const int q_head = head * p.group + row - t * p.group;
  // keys this row sees: [see_lo, see_hi)
  const int see_hi = row_ok ? start + t + 1 : 0;
  const int see_lo = p.window > 0 ? max(start + t - p.window + 1, 0) : 0;
  // keys the tile sees, those of the split among them, and their steps
  const int t_first = nth * kAttnRows / p.group;
  const int t_last = (min(rows, (nth + 1) * kAttnRows) - 1) / p.group;
  const int all_hi = max(start + t_last + 1, 0);
  const int all_lo = p.window > 0 ? max(start + t_first - p.window + 1, 0) : 0;
  const kv::Range range = kv::split_range(split, p.splits, p.chunk, all_lo, all_hi);
  if (range.lo >= range.hi && p.splits > 1) return;       // not joined either
  const int first = range.lo / kStep;
  const int last = (range.hi + kStep - 1) / kStep;

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

  // Loads: a half step's 16 keys lie in one page, so addresses are scalar up
  // to the lane's fixed offset.
  const int head_bytes = kv.dim << kv.page_shift;
  const int8_t* const base = kv.data + long(head) * head_bytes;
  const long v_from = long(kv.kv_heads) * head_bytes;
  const int32_t* const table = kv.table + long(b) * kv.table_ld;
  const int slot_mask = (1 << kv.page_shift) - 1;
  const unsigned k_off = unsigned(r16 * kv.dim + quarter * kQuarter);
  const unsigned v_off = unsigned(quarter * 4 * kv.dim + r16 * kCols);
  auto fetch_pages = [&](int st, int (&page)[2]) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int key = min(st * kStep + 16 * u, range.hi - 1);
      page[u] = kv::scalar_load(table + (max(key, 0) >> kv.page_shift));
    }
  };
  auto fetch = [&](int st, const int (&page)[2], Step<DP>& to) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int key = st * kStep + 16 * u;
      to.ok[u] = key < range.hi && page[u] >= 0 && page[u] < kv.num_pages;
      const long at = to.ok[u] ? page[u] : 0;
      const int8_t* from = base + at * kv.page_stride;
      const int slot = (key & slot_mask) * kv.dim;
      const auto kr = tile::make_rsrc(from, uint32_t(head_bytes));
      const auto vr = tile::make_rsrc(from + v_from, uint32_t(head_bytes));
#pragma unroll
      for (int c = 0; c < DP / 64; ++c) {
        to.k[u][c] = u32x4{0, 0, 0, 0};
        if (!PAD || quarter * kQuarter + 16 * c < kv.dim)
          to.k[u][c] = __builtin_amdgcn_raw_buffer_load_b128(kr, k_off + 16 * c, slot, 0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t (&w)[kVDwords] = to.v[4 * u + i];
        if (PAD) __builtin_memset(w, 0, sizeof(w));
        if (!PAD || r16 * kCols < kv.dim) {
          const int row_at = slot + i * kv.dim;
          if constexpr (kVDwords == 1) {
            w[0] = __builtin_amdgcn_raw_buffer_load_b32(vr, v_off, row_at, 0);
          } else if constexpr (kVDwords == 2) {
            const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(vr, v_off, row_at, 0);
            w[0] = x[0], w[1] = x[1];
          } else {
            const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(vr, v_off, row_at, 0);
            w[0] = x[0], w[1] = x[1], w[2] = x[2], w[3] = x[3];
          }
        }
      }
      const uint16_t* sc = kv.scale + at * kv.scale_stride + head;
      to.sk[u] = sc[0];
      to.sv[u] = sc[kv.kv_heads];
    }
  };

  f32x4 o[kCols];
#pragma unroll
  for (int j = 0; j < kCols; ++j) o[j] = f32x4{0, 0, 0, 0};
  float m = kNone, l = 0.0f;

  auto use = [&](int st, const Step<DP>& in) {
    const int key0 = st * kStep;
    // scores, with the scales of their page
    float x[8], rv[2];
    bool zero[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float sk = key_scale(in.sk[u]) * p.scale_log2e * kCodeScale;
      // an all-zero page has scale 0: for its weights any positive value does,
      // and the smallest leaves the running maximum to the other pages
      const float sv = h2f(uint16_t(in.sv[u]));
      zero[u] = sv == 0.0f;
      const float sv1 = zero[u] ? 0x1p-24f : sv;
      const float lv = __builtin_amdgcn_logf(sv1);
      rv[u] = __builtin_amdgcn_rcpf(sv1);
      f32x4 acc = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < kKStep; ++i)
        acc = mfma16(codes8(biased(in.k[u][i / 2][2 * (i % 2)]), biased(in.k[u][i / 2][2 * (i % 2) + 1])),
                     q[i], acc);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = key0 + 16 * u + quarter * 4 + i;
        const bool seen = in.ok[u] && key >= see_lo && key < see_hi;
        x[4 * u + i] = seen ? __builtin_fmaf(acc[i], sk, lv) : -__builtin_inff();
      }
    }
    float mx = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) mx = fmaxf(mx, x[i]);
    // a row moves its maximum only when a weight would leave fp16's range
    if (__ballot(mx - m > kRoom)) {
      const float m_new = fmaxf(m, lifted(row_max(mx)));
      const float alpha = __builtin_amdgcn_exp2f(m - m_new);
      m = m_new;
      l *= alpha;
#pragma unroll
      for (int j = 0; j < kCols; ++j) o[j] *= alpha;
    }
    half8_t pt;
    float sum[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float e = __builtin_amdgcn_exp2f(x[i] - m);
      sum[i >> 2] += e;
      // whatever the codes of a page with scale 0 are, its values are 0
      pt[i] = static_cast<_Float16>(zero[i >> 2] ? 0.0f : e);
    }
    // a sum of 0 (nothing seen) stays 0 whatever the page's scale holds
#pragma unroll
    for (int u = 0; u < 2; ++u) l += sum[u] == 0.0f ? 0.0f : sum[u] * rv[u];
    // values: 8 keys x kCols columns
#pragma unroll
    for (int c = 0; c < kVDwords; ++c) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = biased(in.v[i][c]);
#pragma unroll
      for (int col = 0; col < 4; ++col) {
        half8_t a;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const half2_t two = codes2(pair_bytes(w[i], w[i + 1], col));
          a[i] = two[0];
          a[i + 1] = two[1];
        }
        o[4 * c + col] = mfma16(a, pt, o[4 * c + col]);
      }
    }
  };

  // One step at a time, with the pages of the next asked for before: four
  // waves a SIMD cover the loads (two steps in flight take the registers of
  // half the waves: 16 x 64 heads x 4000 keys 188 us against 167).
  {
    Step<DP> now;
    int page[2];
    int st = first + wave;
    if (st < last) fetch_pages(st, page);
    while (st < last) {
      fetch(st, page, now);
      fetch_pages(st + kWaves, page);
      if (st == first + wave) {       // here, so that the first keys are asked for before
#pragma unroll
        for (int i = 0; i < kKStep; ++i) q[i] = query8(q[i]);
      }
      use(st, now);
      st += kWaves;
    }
  }
  l = row_sum(l);

  // O^T tile j: lane holds result rows 4 quarter + i, i.e. columns
  // (4 quarter + i) * kCols + j of its row.  Join the four waves through LDS.
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
  // wave w finishes result row i = w of each quarter: kCols columns
  const int d0 = (4 * quarter + wave) * kCols;
  if (PAD && d0 >= kv.dim) return;
  float out[kCols];
#pragma unroll
  for (int j = 0; j < kCols; ++j) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += sh_o[w][lane][j][wave] * factor[w];
    out[j] = v;
  }
  if (p.splits == 1) {
    const float norm = l_all > 0.0f || l_all != l_all ? kCodeScale / l_all : 0.0f;
    uint16_t* dst = p.out + long(s.lo + t) * p.ldo + long(q_head) * kv.dim + d0;
#pragma unroll
    for (int j = 0; j < kCols; ++j) dst[j] = f2h_bits(out[j] * norm);
  } else {
    const long at = (long(s.lo + t) * p.q_heads + q_head) * p.splits + split;
    if (quarter == 0 && wave == 0) p.part_ml[at] = make_float2(m_all, l_all);
    float4* dst = reinterpret_cast<float4*>(p.part_o + at * kv.dim + d0);
#pragma unroll
    for (int j = 0; j < kCols; j += 4) dst[j / 4] = make_float4(out[j], out[j + 1], out[j + 2], out[j + 3]);
  }
}

// The splits of a row, joined in a fixed order of sums.  WPR waves share a
// row; each takes 64 / (dim / 4) splits at a time, dim / 4 lanes a split.
template <int WPR>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnParams p) {
  const KvArgs& kv = p.kv;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const long row = WPR == 1 ? long(blockIdx.x) * 4 + wave : long(blockIdx.x);
  const bool row_ok = row < long(kv.total_q) * p.q_heads;
  const int t = row_ok ? int(row / p.q_heads) : 0;
  const int q_head = int(row - long(t) * p.q_heads);
  int b = t, nth = 0;
  if (kv.cu_q) b = kv::owner(t, kv.batch, [&](int i) { return kv.cu_q[i]; }, &nth);
  const kv::Seq s = kv::seq_of(kv, b);
  // the splits that hold keys of this row
  const int see_hi = max(s.len - s.hi + t + 1, 0);
  const int see_lo = p.window > 0 ? max(see_hi - p.window, 0) : 0;
  const int s0 = min(see_lo / p.chunk, p.splits - 1);
  const int s1 = row_ok && see_hi > 0 ? min((see_hi - 1) / p.chunk, p.splits - 1) + 1 : s0;

  const float2* ml = p.part_ml + row * p.splits;
  const float* part = p.part_o + row * p.splits * kv.dim;
  float m = kNone;
  for (int i = s0 + lane; i < s1; i += 64) m = fmaxf(m, ml[i].x);
#pragma unroll
  for (int x = 32; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor(m, x));
  const int per = kv.dim >> 2;                  // lanes of a split
  const int groups = 64 / per;                  // splits of a wave at once
  const int g = lane / per, d = (lane - g * per) * 4;
  const int team = WPR == 1 ? 0 : wave;
  float4 sum = {0, 0, 0, 0};
  float l = 0.0f;
  if (g < groups) {
#pragma unroll 4
    for (int i = s0 + team * groups + g; i < s1; i += WPR * groups) {
      const float2 a = ml[i];
      const float4 v = *reinterpret_cast<const float4*>(part + long(i) * kv.dim + d);
      const float f = __builtin_amdgcn_exp2f(a.x - m);
      l += a.y * f;
      sum.x += v.x * f;
      sum.y += v.y * f;
      sum.z += v.z * f;
      sum.w += v.w * f;
    }
  }
  __shared__ float4 sh_sum[4][64];
  __shared__ float sh_l[4][64];
  sh_sum[wave][lane] = sum;
  sh_l[wave][lane] = l;
  __syncthreads();
  if (!row_ok || lane >= per || (WPR > 1 && wave > 0)) return;
  float4 all = {0, 0, 0, 0};
  float l_all = 0.0f;
  for (int w = 0; w < WPR; ++w)
    for (int i = 0; i < groups; ++i) {
      const float4 v = sh_sum[WPR == 1 ? wave : w][i * per + lane];
      all.x += v.x;
      all.y += v.y;
      all.z += v.z;
      all.w += v.w;
      l_all += sh_l[WPR == 1 ? wave : w][i * per + lane];
    }
  const float norm = l_all > 0.0f || l_all != l_all ? kCodeScale / l_all : 0.0f;
  uint2 w;
  w.x = f2h_bits(all.x * norm) | uint32_t(f2h_bits(all.y * norm)) << 16;
  w.y = f2h_bits(all.z * norm) | uint32_t(f2h_bits(all.w * norm)) << 16;
  *reinterpret_cast<uint2*>(p.out + long(t) * p.ldo + long(q_head) * kv.dim + d) = w;
}

}  // namespace

hipError_t launch_paged_attn(const AttnParams& p, hipStream_t stream) {
  AttnParams a = p;
  void* args[] = {&a};
  const long wgs = attn_tiles(p.kv, p.group, kAttnRows) * p.kv.kv_heads * p.splits;
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
  // few rows: four waves read a row's splits together
  const long rows = long(p.kv.total_q) * p.q_heads;
  const bool few = rows <= kJoinFewRows;
  const void* fn = few ? reinterpret_cast<const void*>(&attn_join_kernel<4>)
                       : reinterpret_cast<const void*>(&attn_join_kernel<1>);
  return hipLaunchKernel(fn, dim3(unsigned(few ? rows : (rows + 3) / 4)), dim3(256), args, 0, stream);
}

}  // namespace w4a8
