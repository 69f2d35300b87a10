// Attention over the paged int8 cache for many query rows (gfx950): prompts
// and chunks of new tokens.
//
// Rows are (token, query head of the group) pairs as in paged_attn.hip; a
// workgroup of NW waves takes 32 NW of them, 32 a wave, and walks the keys 64
// at a time.  Keys and values are loaded once per workgroup as int8, turned
// to fp16 in registers and staged in LDS, values transposed, two tiles deep:
// while a tile is used, the next one is converted into the other buffer and
// the one after is on its way from memory.
//
// Both products are transposed (v_mfma_f32_32x32x16_f16):
//   S^T[key, row] = K Q^T,   O^T[d, row] += V^T P^T,
// so a lane's accumulators belong to one row (lane % 32), the softmax needs
// one exchange (with lane ^ 32), and P^T's registers are the second
// product's operand as they are: half h of the wave holds keys 8 (i / 4) +
// 4 h + i % 4 of a 32-key score tile, so V^T is staged with the keys of each
// 16 in the order 0-3, 8-11, 4-7, 12-15, half h's 8 keys together.

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

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kKeys = 64;     // keys of a tile
constexpr int kGroups = kKeys / 16;

// Weights above 2^kRoom make a row move its maximum (fp16 ends at 2^16).
constexpr float kRoom = 15.0f;

__device__ __forceinline__ f32x16 mfma32(half8_t a, half8_t b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// what lane ^ 32 holds, combined with the lane's own
__device__ __forceinline__ float pair_max(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__builtin_bit_cast(float, uint32_t(s[0])), __builtin_bit_cast(float, uint32_t(s[1])));
}
__device__ __forceinline__ float pair_sum(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_bit_cast(float, uint32_t(s[0])) + __builtin_bit_cast(float, uint32_t(s[1]));
}

// LDS places, in 16-byte chunks of 8 halves.  A column of chunks is read by
// 32 lanes of consecutive rows; the row-dependent exclusive or spreads 8
// neighbouring rows over all banks (and, for values, the 4-row steps of
// the transposing writes).
template <int DP>
__device__ __forceinline__ int k_chunk(int key, int c) {
  return key * (DP / 8) + (c ^ (key & (DP / 8 - 1) & 15));
}
__device__ __forceinline__ int v_chunk(int d, int c) {
  return d * (kKeys / 8) + (c ^ ((d ^ (d >> 3)) & 7));
}

struct GroupScale {   // of 16 keys
  float sk, lv, rv, pad;
};

template <int DP, bool PAD, int NW>
__global__ __launch_bounds__(64 * NW, DP == 128 ? 2 : 1) void attn_tile_kernel(AttnParams p) {
  constexpr int kThreads = 64 * NW;
  constexpr int kRows = 32 * NW;
  constexpr int kSteps = DP / 16;                       // products of a score tile
  constexpr int kDTiles = DP / 32;
  constexpr int kUnits = kKeys * DP / 16 / kThreads;    // 16-code units of a thread, K and V each
  static_assert(kUnits * kThreads * 16 == kKeys * DP, "units divide evenly");
  const KvArgs& kv = p.kv;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r32 = lane & 31, h = lane >> 5;

  __shared__ half8_t sh_k[2][kKeys * DP / 8];
  __shared__ half8_t sh_v[2][DP * kKeys / 8];
  __shared__ GroupScale sh_s[2][kGroups];

  // heads fastest (neighbouring workgroups land on different dies, so a die
  // keeps few heads' keys in its L2); the last tiles, which see the most
  // keys, first
  const int split = blockIdx.x % p.splits;
  const int rest = blockIdx.x / p.splits;
  const int head = rest % kv.kv_heads;
  const int tiles = gridDim.x / p.splits / kv.kv_heads;
  const int tile = tiles - 1 - rest / kv.kv_heads;
  int b, nth;
  if (kv.cu_q) {
    b = kv::owner(tile, kv.batch,
                  [&](int i) { return int(long(kv.cu_q[i]) * p.group / kRows) + i; }, &nth);
  } else {
    const int per = (p.group + kRows - 1) / kRows;
    b = tile / per;
    nth = tile - b * per;
  }
  const kv::Seq s = kv::seq_of(kv, b);
  const int rows = (s.hi - s.lo) * p.group;
  if (nth < 0 || long(nth) * kRows >= rows) return;     // the whole workgroup
  const int start = s.len - (s.hi - s.lo);              // position of the first new token
  const int row = nth * kRows + wave * 32 + r32;
  const bool row_ok = row < rows;
  const int t = min(row, rows - 1) / p.group;
  const int q_head = head * p.group + min(row, rows - 1) - t * p.group;
  // keys the row sees
  const int see_hi = row_ok ? start + t + 1 : 0;
  const int see_lo = p.window > 0 ? max(start + t - p.window + 1, 0) : 0;
  // keys the workgroup's rows see, and the wave's
  const int wg_t0 = nth * kRows / p.group, wg_t1 = (min(rows, (nth + 1) * kRows) - 1) / p.group;
  const int all_hi = max(start + wg_t1 + 1, 0);
  const int all_lo = p.window > 0 ? max(start + wg_t0 - p.window + 1, 0) : 0;
  const int w_row0 = min(nth * kRows + wave * 32, rows), w_row1 = min(w_row0 + 32, rows);
  const bool w_any = w_row0 < w_row1;
  const int w_t0 = w_any ? w_row0 / p.group : 0, w_t1 = w_any ? (w_row1 - 1) / p.group : 0;
  const int w_hi = w_any ? start + w_t1 + 1 : 0;                          // some row sees below this
  const int w_lo = p.window > 0 ? max(start + w_t0 - p.window + 1, 0) : 0;
  const int w_all_hi = w_any && w_row1 - w_row0 == 32 ? start + w_t0 + 1 : 0;   // every row does
  const int w_all_lo = p.window > 0 ? max(start + w_t1 - p.window + 1, 0) : 0;

  const int tile0 = all_lo / kKeys;
  const int n_tiles = max((all_hi + kKeys - 1) / kKeys - tile0, 0);
  const int first = tile0 + int(long(n_tiles) * split / p.splits);
  const int last = tile0 + int(long(n_tiles) * (split + 1) / p.splits);

  // Q^T: the lane's row, d = 16 i + 8 h ..; a negative score scale turns
  // the queries instead, so that the factors of the scores are >= 0
  half8_t q[kSteps];
  {
    const uint16_t* src = p.q + long(s.lo + t) * p.ldq + long(q_head) * kv.dim;
    const uint32_t flip = p.scale_log2e < 0 ? 0x80008000u : 0u;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int d = 16 * i + 8 * h;
      uint4 u = {0, 0, 0, 0};
      if (row_ok && (!PAD || d < kv.dim)) {
        u = *reinterpret_cast<const uint4*>(src + d);
        u.x ^= flip, u.y ^= flip, u.z ^= flip, u.w ^= flip;
      }
      q[i] = __builtin_bit_cast(half8_t, u);
    }
  }
  const float factor = fabsf(p.scale_log2e) * kCodeScale;

  // A thread's units.  Keys: unit = (key, 16 codes of it).  Values: 4 keys
  // x 4 columns.
  const long head_bytes = long(kv.dim) << kv.page_shift;
  const int slot_mask = (1 << kv.page_shift) - 1;
  uint4 kreg[kUnits], vreg[kUnits];
  int kpage[kUnits], vpage[kUnits];
  int gpage = -1, gthere = -1;           // threads below kGroups: a group's page
  uint16_t gsk = 0, gsv = 0;             // and its scales

  auto k_key = [&](int u) { return (tid + u * kThreads) / (DP / 16); };
  auto k_d = [&](int u) { return (tid + u * kThreads) % (DP / 16) * 16; };
  auto v_kg = [&](int u) { return (tid + u * kThreads) / (DP / 4); };
  auto v_d = [&](int u) { return (tid + u * kThreads) % (DP / 4) * 4; };
  auto page_of = [&](int key) {
    return key < all_hi ? max(kv::page_at(kv, b, key >> kv.page_shift), 0) : 0;
  };
  auto load_pages = [&](int tl) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      kpage[u] = page_of(tl * kKeys + k_key(u));
      vpage[u] = page_of(tl * kKeys + v_kg(u) * 4);
    }
    if (tid < kGroups) {
      const int key = tl * kKeys + tid * 16;
      gpage = key < all_hi ? kv::page_at(kv, b, key >> kv.page_shift) : -1;
    }
  };
  auto load_tile = [&](int tl) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int key = tl * kKeys + k_key(u), d = k_d(u);
      const int8_t* src = kv.data + long(kpage[u]) * kv.page_stride + head * head_bytes +
                          long(key & slot_mask) * kv.dim + d;
      kreg[u] = uint4{0, 0, 0, 0};
      if (!PAD || d < kv.dim) kreg[u] = *reinterpret_cast<const uint4*>(src);
      const int vkey = tl * kKeys + v_kg(u) * 4, vd = v_d(u);
      const int8_t* vs = kv.data + long(vpage[u]) * kv.page_stride +
                         (kv.kv_heads + head) * head_bytes + long(vkey & slot_mask) * kv.dim + vd;
      vreg[u] = uint4{0, 0, 0, 0};
      if (!PAD || vd < kv.dim) {
        vreg[u].x = *reinterpret_cast<const uint32_t*>(vs);
        vreg[u].y = *reinterpret_cast<const uint32_t*>(vs + kv.dim);
        vreg[u].z = *reinterpret_cast<const uint32_t*>(vs + 2 * kv.dim);
        vreg[u].w = *reinterpret_cast<const uint32_t*>(vs + 3 * kv.dim);
      }
    }
    if (tid < kGroups) {
      gthere = gpage;
      const uint16_t* sc = kv.scale + long(max(gpage, 0)) * kv.scale_stride + head;
      gsk = sc[0];
      gsv = sc[kv.kv_heads];
    }
  };
  auto stage_tile = [&](int buf) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int key = k_key(u), c = k_d(u) / 8;
      sh_k[buf][k_chunk<DP>(key, c)] = codes8(biased(kreg[u].x), biased(kreg[u].y));
      sh_k[buf][k_chunk<DP>(key, c + 1)] = codes8(biased(kreg[u].z), biased(kreg[u].w));
      const int kg = v_kg(u), d = v_d(u), g = kg & 3;
      const int c2 = (kg >> 2) * 2 + (g & 1);
      const uint32_t w0 = biased(vreg[u].x), w1 = biased(vreg[u].y), w2 = biased(vreg[u].z),
                     w3 = biased(vreg[u].w);
#define W4A8_COLUMN(B)                                                                   \
  {                                                                                      \
    typedef _Float16 half4_t __attribute__((ext_vector_type(4)));                        \
    const half2_t lo = codes2(pair_bytes<B>(w0, w1)), hi = codes2(pair_bytes<B>(w2, w3)); \
    half4_t four = {lo[0], lo[1], hi[0], hi[1]};                                         \
    reinterpret_cast<half4_t*>(&sh_v[buf][v_chunk(d + B, c2)])[g >> 1] = four;           \
  }
      W4A8_COLUMN(0)
      W4A8_COLUMN(1)
      W4A8_COLUMN(2)
      W4A8_COLUMN(3)
#undef W4A8_COLUMN
    }
    if (tid < kGroups) {
      // a group that is not there has weights exp2(-inf) = 0
      GroupScale g = {0.0f, -__builtin_inff(), 0.0f, 0.0f};
      if (gthere >= 0) {
        const float sv = h2f(gsv);
        const float sv1 = sv == 0.0f ? 0x1p-24f : sv;   // as in paged_attn.hip
        g.sk = h2f(gsk) * factor;
        g.lv = __builtin_amdgcn_logf(sv1);
        g.rv = __builtin_amdgcn_rcpf(sv1);
      }
      sh_s[buf][tid] = g;
    }
  };

  f32x16 o[kDTiles];
#pragma unroll
  for (int j = 0; j < kDTiles; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[j][i] = 0.0f;
  float m = kNone, l = 0.0f;

  if (first < last) {
    load_pages(first);
    load_tile(first);
    load_pages(first + 1);
    stage_tile(0);
    load_tile(first + 1);
    load_pages(first + 2);
  }
  __syncthreads();
  for (int tl = first; tl < last; ++tl) {
    const int buf = (tl - first) & 1;
    if (tl + 1 < last) {
      stage_tile(buf ^ 1);
      load_tile(tl + 2);
      load_pages(tl + 3);
    }
    const int key0 = tl * kKeys;
    if (key0 < w_hi && key0 + kKeys > w_lo) {           // some row of the wave sees some key
      f32x16 acc[2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[u][i] = 0.0f;
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          acc[u] = mfma32(sh_k[buf][k_chunk<DP>(32 * u + r32, 2 * i + h)], q[i], acc[u]);

      GroupScale g[kGroups];
#pragma unroll
      for (int i = 0; i < kGroups; ++i) g[i] = sh_s[buf][i];
      if (key0 + kKeys > w_all_hi || key0 < w_all_lo) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int key = key0 + 32 * u + 8 * (i >> 2) + 4 * h + (i & 3);
            const GroupScale& gs = g[2 * u + (i >> 3)];
            // a key that is not seen is gone here, whatever its page's scale
            acc[u][i] = key >= see_lo && key < see_hi ? __builtin_fmaf(acc[u][i], gs.sk, gs.lv)
                                                      : -__builtin_inff();
          }
#pragma unroll
        for (int n = 0; n < kGroups; ++n) g[n].sk = 1.0f, g[n].lv = 0.0f;
      }
      // the row's largest score: within 16 keys the largest product's, as
      // the factor is >= 0
      float mx = -__builtin_inff();
#pragma unroll
      for (int n = 0; n < kGroups; ++n) {
        float top = acc[n >> 1][8 * (n & 1)];
#pragma unroll
        for (int i = 1; i < 8; ++i) top = fmaxf(top, acc[n >> 1][8 * (n & 1) + i]);
        mx = fmaxf(mx, __builtin_fmaf(top, g[n].sk, g[n].lv));
      }
      mx = pair_max(mx);
      if (__ballot(mx > m + kRoom)) {
        const float m_new = fmaxf(m, mx - kLift);
        const float alpha = __builtin_amdgcn_exp2f(m - m_new);
        m = m_new;
        l *= alpha;
#pragma unroll
        for (int j = 0; j < kDTiles; ++j) o[j] *= alpha;
      }
      half8_t pt[kGroups];
#pragma unroll
      for (int n = 0; n < kGroups; ++n) {
        const float c = g[n].lv - m;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[n >> 1][8 * (n & 1) + i], g[n].sk, c));
          sum += e;
          pt[n][i] = static_cast<_Float16>(e);
        }
        l += sum == 0.0f ? 0.0f : sum * g[n].rv;
      }
#pragma unroll
      for (int n = 0; n < kGroups; ++n)
#pragma unroll
        for (int j = 0; j < kDTiles; ++j)
          o[j] = mfma32(sh_v[buf][v_chunk(32 * j + r32, 2 * n + h)], pt[n], o[j]);
    }
    __syncthreads();
  }
  l = pair_sum(l);
  if (!row_ok) return;

  // o[j][i] is column 32 j + 8 (i / 4) + 4 h + i % 4 of the lane's row
  if (p.splits == 1) {
    const float norm = l > 0.0f || l != l ? kCodeScale / l : 0.0f;
    uint16_t* dst = p.out + long(s.lo + t) * p.ldo + long(q_head) * kv.dim;
#pragma unroll
    for (int j = 0; j < kDTiles; ++j)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int d = 32 * j + 2 * i + 4 * h;
        if (PAD && d >= kv.dim) continue;
        uint2 w;
        w.x = f2h_bits(o[j][i] * norm) | uint32_t(f2h_bits(o[j][i + 1] * norm)) << 16;
        w.y = f2h_bits(o[j][i + 2] * norm) | uint32_t(f2h_bits(o[j][i + 3] * norm)) << 16;
        *reinterpret_cast<uint2*>(dst + d) = w;
      }
  } else {
    float* dst = p.part + ((long(s.lo + t) * p.q_heads + q_head) * p.splits + split) * (kv.dim + 2);
    if (h == 0) {
      dst[0] = l;
      dst[1] = m;
    }
#pragma unroll
    for (int j = 0; j < kDTiles; ++j)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int d = 32 * j + 8 * (i >> 2) + 4 * h + (i & 3);
        if (!PAD || d < kv.dim) dst[2 + d] = o[j][i];
      }
  }
}

}  // namespace

hipError_t launch_paged_attn_tile(const AttnParams& p, int waves, hipStream_t stream) {
  AttnParams a = p;
  void* args[] = {&a};
  const int dim = p.kv.dim;
  if (waves != 4 && !(waves == 8 && dim > 64 && dim <= 128)) return hipErrorInvalidValue;
  const long wgs = attn_tiles(p.kv, p.group, 32 * waves) * p.kv.kv_heads * p.splits;
  if (wgs > 2147483647l) return hipErrorInvalidValue;
  const void* fn;
  if (dim <= 64)
    fn = dim == 64 ? reinterpret_cast<const void*>(&attn_tile_kernel<64, false, 4>)
                   : reinterpret_cast<const void*>(&attn_tile_kernel<64, true, 4>);
  else if (dim > 128)
    fn = dim == 256 ? reinterpret_cast<const void*>(&attn_tile_kernel<256, false, 4>)
                    : reinterpret_cast<const void*>(&attn_tile_kernel<256, true, 4>);
  else if (waves == 8)
    fn = dim == 128 ? reinterpret_cast<const void*>(&attn_tile_kernel<128, false, 8>)
                    : reinterpret_cast<const void*>(&attn_tile_kernel<128, true, 8>);
  else
    fn = dim == 128 ? reinterpret_cast<const void*>(&attn_tile_kernel<128, false, 4>)
                    : reinterpret_cast<const void*>(&attn_tile_kernel<128, true, 4>);
  return hipLaunchKernel(fn, dim3(unsigned(wgs)), dim3(64 * waves), args, 0, stream);
}

}  // namespace w4a8
