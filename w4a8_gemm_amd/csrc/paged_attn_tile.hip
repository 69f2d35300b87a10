// Attention over the paged int8 cache for many query rows (gfx950): prompts
// and chunks of new tokens.
//
// Rows are (token, query head of the group) pairs as in paged_attn.hip; a
// workgroup of NW waves takes 32 NW of them, 32 a wave, and walks the keys 64
// at a time.  Keys and values are loaded once per workgroup as int8, turned
// to fp16 in registers and staged in LDS, values transposed, two tiles deep.
//
// Both products are transposed (v_mfma_f32_32x32x16_f16):
//   S^T[key, row] = K Q^T,   O^T[d, row] += V^T P^T,
// so a lane's accumulators belong to one row (lane % 32), the softmax needs
// one exchange (with lane ^ 32), and P^T's registers are the second
// product's operand as they are: half h of the wave holds keys 8 (i / 4) +
// 4 h + i % 4 of a 32-key score tile, so V^T is staged with the keys of each
// 16 in the order 0-3, 8-11, 4-7, 12-15, half h's 8 keys together.
//
// Bound by the matrix and vector instructions of a tile (per wave and 64 keys
// 1024 cycles of products, about 700 of softmax and 250 of staging) and the
// first LDS reads after each barrier, some 500 cycles under load.  Measured: a
// prompt of 8192 tokens, 32 + 8 heads of 128, 580 to 610 us = 0.90 to 0.95
// PFLOP/s of the causal half (a library's fp16 matrix product 8192^3 reaches
// 1.15).  Where the tiles are few, the time is that of the longest chain of key
// tiles in a workgroup, 2 us a tile with one workgroup on a unit: 12 ragged
// chunks of up to 200 tokens over a window of 1024 64 us, a prompt of 2000 tokens
// 71, 16 x up to 64 tokens over 2048 keys 76.
// 128 rows a workgroup instead of 256 take 640 us on the prompt, but 67
// against 98 us on the chunks, which 256 rows leave on too few units.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attn_common.h"
#include "decoder_kernels.h"
#include "kv_page.h"
#include "quant_common.h"
#include "tile_common.h"

namespace w4a8 {
namespace {

using namespace attn;
using namespace dev;

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// A lane's weights of a tile may add up to this (fp16 ends at 65504; a weight
// beyond it is infinite, and so is the sum).
constexpr float kMost = 65000.0f;

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

// LDS places, in bytes.  Rows of keys hold DP halves, rows of V^T (one per
// column d) KEYS halves, in 16-byte chunks.  A column of chunks is read by 32
// lanes of consecutive rows, so the row number is spread over the banks by an
// exclusive or on the chunk number: 8 neighbouring rows take all banks, and so
// do, for V^T, the 4-row steps of the transposing writes.
template <int DP>
__device__ __forceinline__ int k_place(int key, int c) {
  return key * (DP * 2) + ((c ^ (key & (DP / 8 - 1) & 15)) << 4);
}
template <int KEYS>
__device__ __forceinline__ int v_place(int d, int c) {
  const int f = KEYS == 64 ? (d ^ (d >> 3)) & 7 : ((d >> 1) ^ (d >> 3)) & 3;
  return d * (KEYS * 2) + ((c ^ f) << 4);
}

struct GroupScale {   // of 16 keys
  float sk, lv, rv;
  float zero;         // 1: the value scale is 0, else 0
};

// Barrier of the workgroup that makes LDS writes visible and, unlike
// __syncthreads, leaves loads from memory in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// DP: head dim rounded up to 64, 128 or 256 (PAD: dim < DP); NW waves; SUB
// 32-key subtiles per staged tile.
template <int DP, bool PAD, int NW, int SUB>
__global__ __launch_bounds__(64 * NW, DP == 256 ? 1 : 2) void attn_tile_kernel(AttnParams p) {
  constexpr int kThreads = 64 * NW;
  constexpr int kRows = 32 * NW;
  constexpr int kKeys = 32 * SUB;
  constexpr int kGroups = kKeys / 16;
  constexpr int kSteps = DP / 16;                       // products of a score subtile
  constexpr int kDTiles = DP / 32;
  constexpr int kUnits = kKeys * DP / 16 / kThreads;    // 16-code units of a thread, K and V each
  constexpr int kWaveKeys = 1024 / DP;                  // keys of a wave's unit: within 16 aligned ones
  constexpr int kUnitKeys = kThreads * 16 / DP;         // keys from one unit of a thread to the next
  static_assert(kUnits * kThreads * 16 == kKeys * DP, "units divide evenly");
  static_assert(kUnits == 1 || kUnitKeys % 16 == 0, "the swizzles repeat from unit to unit");
  const KvArgs& kv = p.kv;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r32 = lane & 31, h = lane >> 5;

  // two tiles deep: see the loop
  constexpr int kTileBytes = kKeys * DP * 2;
  __shared__ __attribute__((aligned(1024))) uint8_t sh_k[2 * kTileBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sh_v[2 * kTileBytes];
  __shared__ GroupScale sh_s[2][kGroups];

  // heads fastest (neighbouring workgroups land on different dies, so a die
  // keeps few heads' keys in its L2); the last tiles, which see the most
  // keys, first
  const int rest = blockIdx.x / p.splits;
  const int split = (blockIdx.x % p.splits + (rest >> 2)) % p.splits;   // turned as in paged_attn.hip
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
  // keys that some row of the workgroup sees, that some row of the wave sees,
  // that all 32 see
  const int wg_t0 = nth * kRows / p.group, wg_t1 = (min(rows, (nth + 1) * kRows) - 1) / p.group;
  const int all_hi = max(start + wg_t1 + 1, 0);
  const int all_lo = p.window > 0 ? max(start + wg_t0 - p.window + 1, 0) : 0;
  const int w_row0 = min(nth * kRows + wave * 32, rows), w_row1 = min(w_row0 + 32, rows);
  const bool w_any = w_row0 < w_row1;
  const int w_t0 = w_any ? w_row0 / p.group : 0, w_t1 = w_any ? (w_row1 - 1) / p.group : 0;
  const int w_hi = w_any ? start + w_t1 + 1 : 0;
  const int w_lo = p.window > 0 ? max(start + w_t0 - p.window + 1, 0) : 0;
  const int w_all_hi = w_row1 - w_row0 == 32 ? start + w_t0 + 1 : 0;
  const int w_all_lo = p.window > 0 ? max(start + w_t1 - p.window + 1, 0) : 0;

  const kv::Range range = kv::split_range(split, p.splits, p.chunk, all_lo, all_hi);
  if (range.lo >= range.hi && p.splits > 1) return;     // not joined either
  const int first = range.lo / kKeys, last = (range.hi + kKeys - 1) / kKeys;
  // the tiles among them that some row of the wave sees
  const int w_first = max(first, w_lo / kKeys);
  const int w_last = min(last, (w_hi + kKeys - 1) / kKeys);

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
      q[i] = query8(__builtin_bit_cast(half8_t, u));
    }
  }
  const float factor = fabsf(p.scale_log2e) * kCodeScale;

  // A thread's units.  Keys: unit = (key, 16 codes of it).  Values: 4 keys
  // x 4 columns.  A wave's share of a tile lies in one page, so its address
  // is scalar up to a fixed offset of the lane.
  const long head_bytes = long(kv.dim) << kv.page_shift;
  const int slot_mask = (1 << kv.page_shift) - 1;
  const int8_t* const k_base = kv.data + head * head_bytes;
  const int8_t* const v_base = k_base + kv.kv_heads * head_bytes;
  const int k_lane_key = lane / (DP / 16), k_lane_d = lane % (DP / 16) * 16;
  const int v_lane_key = lane / (DP / 4) * 4, v_lane_d = lane % (DP / 4) * 4;
  const unsigned k_off = unsigned(k_lane_key * kv.dim + k_lane_d);
  const unsigned v_off = unsigned(v_lane_key * kv.dim + v_lane_d);
  const bool k_there = !PAD || k_lane_d < kv.dim, v_there = !PAD || v_lane_d < kv.dim;
  u32x4 kreg[kUnits], vreg[kUnits];
  int kpage[kUnits], vpage[kUnits];      // of the next tiles to load
  int gpage = -1;                        // threads below kGroups: a group's page,
  bool gthere = false;                   // whether it exists,
  uint32_t gsk = 0, gsv = 0;             // and its scales

  // Page numbers are loaded one tile before they are used and looked at only
  // then: a look at once would wait for that load, and with it for all the
  // loads before it.
  const int32_t* const table = kv.table + long(b) * kv.table_ld;
  auto unit_key = [&](int tl, int u) { return tl * kKeys + wave * kWaveKeys + u * kUnitKeys; };
  auto entry_of = [&](int key) {
    return min(max(min(key, all_hi - 1), 0) >> kv.page_shift, kv.max_pages - 1);
  };
  auto exists = [&](int page) { return page >= 0 && page < kv.num_pages; };
  // one page's keys or values of the head, as a buffer
  const int block_bytes = int(head_bytes);
  auto load_k = [&](int tl) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const auto rsrc = tile::make_rsrc(k_base + long(exists(kpage[u]) ? kpage[u] : 0) * kv.page_stride, block_bytes);
      const int at = (unit_key(tl, u) & slot_mask) * kv.dim;
      kreg[u] = u32x4{0, 0, 0, 0};
      if (k_there) kreg[u] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, k_off, at, 0);
    }
  };
  auto load_v = [&](int tl) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const auto rsrc = tile::make_rsrc(v_base + long(exists(vpage[u]) ? vpage[u] : 0) * kv.page_stride, block_bytes);
      const int at = (unit_key(tl, u) & slot_mask) * kv.dim;
      vreg[u] = u32x4{0, 0, 0, 0};
      if (v_there) {
        vreg[u].x = __builtin_amdgcn_raw_buffer_load_b32(rsrc, v_off, at, 0);
        vreg[u].y = __builtin_amdgcn_raw_buffer_load_b32(rsrc, v_off, at + kv.dim, 0);
        vreg[u].z = __builtin_amdgcn_raw_buffer_load_b32(rsrc, v_off, at + 2 * kv.dim, 0);
        vreg[u].w = __builtin_amdgcn_raw_buffer_load_b32(rsrc, v_off, at + 3 * kv.dim, 0);
      }
    }
  };
  auto load_scales = [&](int tl) {
    if (tid < kGroups) {
      gthere = tl * kKeys + tid * 16 < all_hi && exists(gpage);
      const uint16_t* sc = kv.scale + long(gthere ? gpage : 0) * kv.scale_stride + head;
      gsk = sc[0];
      gsv = sc[kv.kv_heads];
    }
  };
  auto load_k_pages = [&](int tl) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) kpage[u] = kv::scalar_load(table + entry_of(unit_key(tl, u)));
  };
  // tl's value pages are its key pages, if kpage is still tl's
  auto load_v_pages = [&](int tl) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) vpage[u] = kpage[u];
    if (tid < kGroups) gpage = table[entry_of(tl * kKeys + tid * 16)];
  };
  const int k_to0 = k_place<DP>(wave * kWaveKeys + k_lane_key, k_lane_d / 8);
  const int k_to1 = k_place<DP>(wave * kWaveKeys + k_lane_key, k_lane_d / 8 + 1);
  // Staging, in parts that fit between matrix instructions: half of a unit's
  // keys, one column of a unit's values.
  auto stage_k_part = [&](int buf, int u, int half) {
    uint8_t* dst = sh_k + buf * kTileBytes + u * kUnitKeys * DP * 2;
    if (half == 0)
      *reinterpret_cast<half8_t*>(dst + k_to0) = codes8(biased(kreg[u].x), biased(kreg[u].y));
    else
      *reinterpret_cast<half8_t*>(dst + k_to1) = codes8(biased(kreg[u].z), biased(kreg[u].w));
  };
  auto stage_v_part = [&](int buf, int u, int col) {
    typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
    const int kg = (wave * kWaveKeys + v_lane_key + u * kUnitKeys) >> 2, g = kg & 3;
    const int c = (kg >> 2) * 2 + (g & 1);
    const uint32_t sel = 0x0c040c00u + 0x00010001u * col;     // byte `col` of two words
    const half2_t lo = codes2(__builtin_amdgcn_perm(biased(vreg[u].y), biased(vreg[u].x), sel));
    const half2_t hi = codes2(__builtin_amdgcn_perm(biased(vreg[u].w), biased(vreg[u].z), sel));
    const half4_t four = {lo[0], lo[1], hi[0], hi[1]};
    *reinterpret_cast<half4_t*>(sh_v + buf * kTileBytes + v_place<kKeys>(v_lane_d + col, c) +
                                8 * (g >> 1)) = four;
  };
  auto stage_k = [&](int buf) {
#pragma unroll
    for (int i = 0; i < 2 * kUnits; ++i) stage_k_part(buf, i >> 1, i & 1);
  };
  auto stage_v = [&](int buf) {
#pragma unroll
    for (int i = 0; i < 4 * kUnits; ++i) stage_v_part(buf, i >> 2, i & 3);
  };
  auto stage_scales = [&](int buf) {
    if (tid < kGroups) {
      // a group that is not there has weights exp2(-inf) = 0
      GroupScale g = {0.0f, -__builtin_inff(), 0.0f, 0.0f};
      if (gthere) {
        const float sv = h2f(uint16_t(gsv));
        const float sv1 = sv == 0.0f ? 0x1p-24f : sv;   // as in paged_attn.hip
        g.zero = sv == 0.0f ? 1.0f : 0.0f;
        g.sk = key_scale(gsk) * factor;
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

  // The matrix instructions of a tile: numbers 0 .. kWeighs - 1 add its
  // values, O^T += V^T P^T, and the kScores after them make the next tile's
  // scores, S^T = K Q^T.  Each reads one LDS operand, kAhead instructions in
  // front; `between(n)` follows instruction n.  The order is fixed here, by
  // barriers to the compiler's scheduler.  The chunk's part of an address is
  // an exclusive or that can follow the buffer's addition (buffers are
  // multiples of 1024 bytes).
  constexpr int kAhead = 6;
  constexpr int kWeighs = kGroups * kDTiles, kScores = kSteps * SUB;
  f32x16 acc[SUB];
  half8_t pt[kGroups];
#pragma unroll
  for (int n = 0; n < kGroups; ++n)
#pragma unroll
    for (int i = 0; i < 8; ++i) pt[n][i] = (_Float16)0.0f;
  const int k_from = k_place<DP>(r32, h), v_from = v_place<kKeys>(r32, h);
  auto products = [&](int v_buf, int k_buf, auto begin, auto end, auto between) {
    constexpr int n0 = decltype(begin)::value, n1 = decltype(end)::value;
    const int vf = v_from + v_buf * kTileBytes, kf = k_from + k_buf * kTileBytes;
    auto read = [&](int n) {
      if (n < kWeighs) {             // 16 keys n / kDTiles, 32 columns n % kDTiles
        const int i = n % kDTiles;
        // 32 columns on, the row's bit 5 turns chunk bit 2 (64-key rows)
        const int turn = (2 * (n / kDTiles) ^ (kKeys == 64 ? 4 * (i & 1) : 0)) << 4;
        return *reinterpret_cast<const half8_t*>(sh_v + (vf ^ turn) + i * 64 * kKeys);
      }
      const int j = n - kWeighs;     // step j / SUB of subtile j % SUB
      return *reinterpret_cast<const half8_t*>(sh_k + (kf ^ (j / SUB << 5)) + j % SUB * 64 * DP);
    };
    half8_t a[kAhead];
#pragma unroll
    for (int n = n0; n < n0 + kAhead; ++n) a[n % kAhead] = read(n);
    f32x16 zero;
#pragma unroll
    for (int e = 0; e < 16; ++e) zero[e] = 0.0f;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = n0; n < n1; ++n) {
      if (n < kWeighs) {
        o[n % kDTiles] = mfma32(a[n % kAhead], pt[n / kDTiles], o[n % kDTiles]);
      } else {
        const int j = n - kWeighs;
        acc[j % SUB] = mfma32(a[n % kAhead], q[j / SUB], j < SUB ? zero : acc[j % SUB]);
      }
      if (n + kAhead < n1) a[n % kAhead] = read(n + kAhead);
      between(n - n0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  using std::integral_constant;
  const integral_constant<int, 0> values_begin;
  const integral_constant<int, kWeighs> scores_begin;
  const integral_constant<int, kWeighs + kScores> scores_end;
  // acc -> pt, and the row's sum.  Weights are taken relative to the maximum
  // the row has (m is it, less kLift); only when a sum shows that one of
  // them may leave fp16's range, the row's maximum is looked for and moved, and
  // the weights are taken again.
  // That happens in the first tile and rarely after, so the usual tile
  // needs no maximum and no exchange between lanes.
  auto soften = [&](int tl, int buf) {
    const int key0 = tl * kKeys;
    GroupScale g[kGroups];
#pragma unroll
    for (int n = 0; n < kGroups; ++n) g[n] = sh_s[buf][n];
    if (key0 + kKeys > w_all_hi || key0 < w_all_lo) {
      // a key that is not seen is gone here, whatever its page's scale
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int key = key0 + 32 * u + 8 * (i >> 2) + 4 * h + (i & 3);
          const GroupScale& gs = g[2 * u + (i >> 3)];
          acc[u][i] = key >= see_lo && key < see_hi ? __builtin_fmaf(acc[u][i], gs.sk, gs.lv)
                                                    : -__builtin_inff();
        }
#pragma unroll
      for (int n = 0; n < kGroups; ++n) {
        const int key = key0 + 16 * n;
        g[n].sk = 1.0f;
        g[n].lv = 0.0f;
        g[n].rv = key < see_hi && key + 16 > see_lo ? g[n].rv : 0.0f;
      }
    }
    float zeros = g[0].zero;
#pragma unroll
    for (int n = 1; n < kGroups; ++n) zeros += g[n].zero;
    float sum[kGroups];
    auto weights = [&](auto again) {
#pragma unroll
      for (int n = 0; n < kGroups; ++n) {
        const float c = g[n].lv - m;
        sum[n] = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // again: as the maximum was found, from the rounded score (a score of
          // 2^27 and its rounding are up to 8 apart)
          const float a = acc[n >> 1][8 * (n & 1) + i];
          const float x = decltype(again)::value ? __builtin_fmaf(a, g[n].sk, g[n].lv) - m
                                                 : __builtin_fmaf(a, g[n].sk, c);
          const float e = __builtin_amdgcn_exp2f(x);
          // summed before the rounding: a weight carries its page's value
          // scale, and where that is far below the others' the rounded weight
          // has few bits or none, while its part of the sum, once the scale is
          // divided out, may be the largest
          sum[n] += e;
          pt[n][i] = static_cast<_Float16>(e);
        }
      }
    };
    weights(std::false_type());
    float most = sum[0];
#pragma unroll
    for (int n = 1; n < kGroups; ++n) most += sum[n];
    if (__ballot(!(most <= kMost))) {
      float mx = -__builtin_inff();
#pragma unroll
      for (int n = 0; n < kGroups; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          mx = fmaxf(mx, __builtin_fmaf(acc[n >> 1][8 * (n & 1) + i], g[n].sk, g[n].lv));
      const float m_new = fmaxf(m, lifted(pair_max(mx)));
      const float alpha = __builtin_amdgcn_exp2f(m - m_new);
      m = m_new;
      l *= alpha;
#pragma unroll
      for (int i = 0; i < kDTiles; ++i) o[i] *= alpha;
      weights(std::true_type());
    }
#pragma unroll
    for (int n = 0; n < kGroups; ++n) l = __builtin_fmaf(sum[n], g[n].rv, l);
    // whatever the codes of a page with scale 0 are, its values are 0
    if (__builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, zeros)) != 0) {
#pragma unroll
      for (int n = 0; n < kGroups; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i) pt[n][i] = g[n].zero != 0.0f ? (_Float16)0.0f : pt[n][i];
    }
  };

  // Each tile is a stretch of vector work (softmax of its scores) and one of
  // matrix work (its values, the next tile's scores), with the staging of
  // later tiles between the matrix instructions.  With 8 waves the second
  // four run one stretch behind the first, so that on every SIMD one wave's
  // products run beside the other's softmax; a barrier after every stretch
  // keeps them in step.
  // At tile t's matrix stretch keys of t + 2 and values of t + 1 are staged,
  // into the buffers of t's keys and t - 1's values, which every wave must
  // have read for the last time:
  //   t's keys are read by the scores of t, in the matrix stretch of t - 1 or,
  //   for the first tile, before the loop; t - 1's values in the stretch of t - 1.
  //   With 8 waves the barriers around the softmax of t lie between (a half's
  //   stretch t - 1 ends two barriers before its stretch t, the other half's
  //   one before it).  With 4 waves the barrier at the end of an iteration
  //   does for t > first, and one of its own after the first scores for
  //   t = first: a wave without rows, or whose window starts later, has no scores
  //   to make there and would reach its staging while others still read.
  // The barrier after the (second half's) stretch comes before anyone reads
  // what was staged.
  constexpr bool kTwoHalves = NW == 8;
  const bool behind = kTwoHalves && wave >= NW / 2;
  if (first < last) {
    load_k_pages(first);
    load_k(first);
    load_v_pages(first);
    load_v(first);
    load_k_pages(first + 1);
    load_scales(first);
    stage_k(0);
    stage_v(0);
    stage_scales(0);
    load_k(first + 1);
    load_v_pages(first + 1);
    load_v(first + 1);
    load_scales(first + 1);
    load_k_pages(first + 2);
    stage_k(1);
    load_k(first + 2);
    load_v_pages(first + 2);
    load_k_pages(first + 3);
  }
  lds_barrier();
  if (w_first == first && w_first < w_last)
    products(0, 0, scores_begin, scores_end, [](int) {});
  if (!kTwoHalves || behind) lds_barrier();
  int buf = 0;
  for (int tl = first; tl < last; ++tl) {
    // asked for first: the barriers wait for scalar loads as well
    int later[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) later[u] = kv::scalar_load(table + entry_of(unit_key(tl + 4, u)));
    const bool mine = tl >= w_first && tl < w_last;
    const bool mine_next = tl + 1 >= w_first && tl + 1 < w_last;
    if (mine) soften(tl, buf);
    if (kTwoHalves) {
      lds_barrier();
      __builtin_amdgcn_s_setprio(1);
    }
    // what goes between: the staging, part by part, and the loads of later
    // tiles, each after its registers are free
    constexpr int kJobs = 6 * kUnits + 4;
    auto job = [&](int i) {
      if (i < 4 * kUnits) stage_v_part(buf ^ 1, i / 4, i % 4);
      else if (i == 4 * kUnits) load_v(tl + 2);
      else if (i <= 6 * kUnits) stage_k_part(buf, (i - 4 * kUnits - 1) / 2, (i - 4 * kUnits - 1) % 2);
      else if (i == 6 * kUnits + 1) load_k(tl + 3);
    };
    if (mine || mine_next) {
      // where only one of them is the wave's, the other half does no harm: the
      // weights are still 0, or the scores are not looked at
      products(buf, buf ^ 1, values_begin, scores_end, [&](int n) {
#pragma unroll
        for (int i = 0; i < kJobs; ++i)
          if (i * (kWeighs + kScores) / kJobs == n) job(i);
      });
    } else {
#pragma unroll
      for (int i = 0; i < kJobs; ++i) job(i);
    }
    stage_scales(buf ^ 1);
    load_scales(tl + 2);
    load_v_pages(tl + 3);
#pragma unroll
    for (int u = 0; u < kUnits; ++u) kpage[u] = later[u];
    if (kTwoHalves) __builtin_amdgcn_s_setprio(0);
    lds_barrier();
    buf ^= 1;
  }
  if (kTwoHalves && !behind) lds_barrier();
  l = pair_sum(l);
  if (!row_ok) return;
  if (l != l) {
    // keys of absent pages have weights exp2(-inf) = 0, but under a query that
    // is not finite NaN: a row that sees no others is nothing all the same
    const int hi = min(see_hi, range.hi);
    bool any = false;
    for (int key = max(see_lo, range.lo) & ~slot_mask; key < hi; key += slot_mask + 1)
      any |= exists(table[key >> kv.page_shift]);
    if (!any) {
      l = 0.0f;
#pragma unroll
      for (int j = 0; j < kDTiles; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[j][i] = 0.0f;
    }
  }

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
    const long at = (long(s.lo + t) * p.q_heads + q_head) * p.splits + split;
    if (h == 0) p.part_ml[at] = make_float2(m, l);
    float* dst = p.part_o + at * kv.dim;
#pragma unroll
    for (int j = 0; j < kDTiles; ++j)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int d = 32 * j + 2 * i + 4 * h;
        if (!PAD || d < kv.dim)
          *reinterpret_cast<float4*>(dst + d) = make_float4(o[j][i], o[j][i + 1], o[j][i + 2], o[j][i + 3]);
      }
  }
}

}  // namespace

hipError_t launch_paged_attn_tile(const AttnParams& p, int waves, hipStream_t stream) {
  AttnParams a = p;
  void* args[] = {&a};
  const int dim = p.kv.dim;
  const long wgs = attn_tiles(p.kv, p.group, 32 * waves) * p.kv.kv_heads * p.splits;
  const void* fn;
  if (dim <= 64)
    fn = dim == 64 ? reinterpret_cast<const void*>(&attn_tile_kernel<64, false, 4, 2>)
                   : reinterpret_cast<const void*>(&attn_tile_kernel<64, true, 4, 2>);
  else if (dim > 128)
    fn = dim == 256 ? reinterpret_cast<const void*>(&attn_tile_kernel<256, false, 4, 1>)
                    : reinterpret_cast<const void*>(&attn_tile_kernel<256, true, 4, 1>);
  else if (waves == 8)
    fn = dim == 128 ? reinterpret_cast<const void*>(&attn_tile_kernel<128, false, 8, 2>)
                    : reinterpret_cast<const void*>(&attn_tile_kernel<128, true, 8, 2>);
  else
    fn = dim == 128 ? reinterpret_cast<const void*>(&attn_tile_kernel<128, false, 4, 2>)
                    : reinterpret_cast<const void*>(&attn_tile_kernel<128, true, 4, 2>);
  return hipLaunchKernel(fn, dim3(unsigned(wgs)), dim3(64 * waves), args, 0, stream);
}

}  // namespace w4a8
