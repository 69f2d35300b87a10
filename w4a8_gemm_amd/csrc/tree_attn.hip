// Attention of drafted token trees over the paged int8 cache (gfx950).
//
// A row is one (drafted token, query head); it sees every cached position
// before the sequence's drafted tokens and those of them that its mask names.
// The rows of a sequence and kv head are few (8 to 200 tokens times the group)
// and the keys many, so nothing is staged: each of a workgroup's four waves
// takes every fourth step of 32 keys straight from memory into registers, turns
// the codes to fp16 once, and uses them for R tiles of 16 rows.  Layouts of both
// products and of the softmax are those of paged_attn.hip:
//   S^T[key, row] = K Q^T,   O^T[d, row] += V^T P^T   (v_mfma_f32_16x16x32_f16)
// The waves join through LDS; where there are few row tiles, the keys are split
// over workgroups as well and attn_join_kernel joins them.

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

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = 32;      // keys a wave takes at once
// A lane's weights of a step may add up to this (fp16 ends at 65504).
constexpr float kMost = 65000.0f;

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// over the four lanes of a row (lane, lane ^ 16, lane ^ 32, ...)
__device__ __forceinline__ float row_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float row_sum(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

// Which of the 32 positions from `at` on, counted from the sequence's first
// drafted token, a row's mask lets it see; those before 0 are cached tokens.
__device__ __forceinline__ uint32_t mask_window(const uint32_t* row, int words, int at) {
  if (at <= -32) return ~0u;
  if (at < 0) return row[0] << -at | ((1u << -at) - 1);
  const int w = at >> 5, shift = at & 31;
  const uint32_t lo = w < words ? row[w] : 0u;
  if (shift == 0) return lo;
  const uint32_t hi = w + 1 < words ? row[w + 1] : 0u;
  return lo >> shift | hi << (32 - shift);
}

// The first position a row sees under a window: the last `window` of the
// positions that its mask names and the cached ones before them.
__device__ __forceinline__ int window_begin(const uint32_t* row, int words, int n, int start,
                                            int window) {
  const int used = min(words, (n + 31) >> 5);
  auto word = [&](int w) {
    const int left = n - 32 * w;
    return left < 32 ? row[w] & ((1u << left) - 1) : row[w];
  };
  int count = 0;
  for (int w = 0; w < used; ++w) count += __builtin_popcount(word(w));
  int drop = count - window;             // drafted tokens that the window leaves out
  if (drop <= 0) return max(start + drop, 0);
  for (int w = 0; w < used; ++w) {
    uint32_t bits = word(w);
    const int here = __builtin_popcount(bits);
    if (drop >= here) {
      drop -= here;
      continue;
    }
    for (; drop > 0; --drop) bits &= bits - 1;
    return start + 32 * w + __builtin_ctz(bits);
  }
  return start + n;
}

// DP: head dim rounded up to 64, 128 or 256.  PAD: dim < DP.  R: row tiles of
// 16 that a workgroup takes; up to 256 query values a lane quarter stay in
// registers, more are read from LDS at each step.
template <int DP, bool PAD, int R>
__global__ __launch_bounds__(kThreads, DP * R > 128 ? 2 : 3) void tree_attn_kernel(AttnParams p) {
  constexpr int kRows = 16 * R;
  constexpr int kQuarter = DP / 4;        // K bytes of a lane and key
  constexpr int kKStep = DP / 32;         // products of one 16-key score tile
  constexpr int kCols = DP / 16;          // V columns of a lane
  constexpr int kVDwords = DP / 64;       // dwords of those columns and one key
  constexpr bool kHeld = DP * R <= 256;
  const KvArgs& kv = p.kv;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, quarter = lane >> 4;

  // splits fastest, turned from row tile to row tile (as in paged_attn.hip)
  const int rest = blockIdx.x / p.splits;
  const int split = (blockIdx.x % p.splits + (rest >> 2)) % p.splits;
  const int head = rest % kv.kv_heads;
  const int tile = rest / kv.kv_heads;
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
  const int n = s.hi - s.lo;
  const int rows = n * p.group;
  if (nth < 0 || long(nth) * kRows >= rows) return;       // the whole workgroup
  const int start = s.len - n;                            // position of the first drafted token
  const int all_lo = p.window > 0 ? max(start - p.window, 0) : 0;
  const kv::Range range = kv::split_range(split, p.splits, p.chunk, all_lo, s.len);
  if (range.lo >= range.hi && p.splits > 1) return;       // not joined either
  const int first = range.lo / kStep;
  const int last = (range.hi + kStep - 1) / kStep;

  // a lane's row of tile j: drafted token and query head.  Worked out again
  // wherever it is needed (the asm hides that it is the same): kept, it would take
  // registers through the whole loop.
  auto row_of = [&](int j, int* t, int* q_head) {
    int first_row = nth * kRows;
    asm volatile("" : "+s"(first_row));
    const int row = first_row + 16 * j + r16;
    const int r = min(row, rows - 1);
    *t = r / p.group;
    *q_head = head * p.group + r - *t * p.group;
    return row < rows;
  };
  int see_lo[R], see_most = 0;                            // see_most: no row starts later
#pragma unroll
  for (int j = 0; j < R; ++j) {
    int t, q_head;
    row_of(j, &t, &q_head);
    see_lo[j] = 0;
    if (p.window > 0)
      see_lo[j] = window_begin(p.mask + long(s.lo + t) * p.mask_ld, p.mask_words, n, start, p.window);
    see_most = max(see_most, see_lo[j]);
  }
  if (p.window > 0) {
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) see_most = max(see_most, __shfl_xor(see_most, x));
    see_most = __builtin_amdgcn_readfirstlane(see_most);
  }

  // LDS: the waves' results at the end and, before, the queries where they are
  // not held
  __shared__ f32x4 sh_o[kWaves][64][kCols + 1];
  static_assert(R * kKStep * 64 * sizeof(half8_t) <= sizeof(sh_o), "the queries fit");
  half8_t (*const sh_q)[64] = reinterpret_cast<half8_t (*)[64]>(&sh_o[0][0][0]);

  // Q^T fragments: lane's row, d = quarter * DP/4 + 8 i ..
  half8_t q[kHeld ? R : 1][kHeld ? kKStep : 1];
  auto load_q = [&](int j, int i) {
    int t, q_head;
    const bool ok = row_of(j, &t, &q_head);
    const int d = quarter * kQuarter + 8 * i;
    uint4 u = {0, 0, 0, 0};
    if (ok && (!PAD || d < kv.dim))
      u = *reinterpret_cast<const uint4*>(p.q + long(s.lo + t) * p.ldq + long(q_head) * kv.dim + d);
    return query8(__builtin_bit_cast(half8_t, u));
  };
  if constexpr (kHeld) {
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int i = 0; i < kKStep; ++i) q[j][i] = load_q(j, i);
  } else {
    for (int j = wave; j < R; j += kWaves)
#pragma unroll
      for (int i = 0; i < kKStep; ++i) sh_q[j * kKStep + i][lane] = load_q(j, i);
    __syncthreads();
  }

  // Loads, as in paged_attn.hip: a half step's 16 keys lie in one page.
  const int head_bytes = kv.dim << kv.page_shift;
  const int8_t* const base = kv.data + long(head) * head_bytes;
  const long v_from = long(kv.kv_heads) * head_bytes;
  const int32_t* const table = kv.table + long(b) * kv.table_ld;
  const int slot_mask = (1 << kv.page_shift) - 1;
  const unsigned k_off = unsigned(r16 * kv.dim + quarter * kQuarter);
  const unsigned v_off = unsigned(quarter * 4 * kv.dim + r16 * kCols);
  int page[2];
  auto fetch_pages = [&](int st) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int key = min(st * kStep + 16 * u, range.hi - 1);
      page[u] = kv::scalar_load(table + (max(key, 0) >> kv.page_shift));
    }
  };
  auto there = [&](int st, int u) {
    return st * kStep + 16 * u < range.hi && page[u] >= 0 && page[u] < kv.num_pages;
  };
  u32x4 kreg[2][DP / 64];
  uint32_t vreg[8][kVDwords];
  uint32_t sk_bits[2], sv_bits[2];
  bool ok[2];
  auto load_k = [&](int st) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      ok[u] = there(st, u);
      const long at = ok[u] ? page[u] : 0;
      const auto rsrc = tile::make_rsrc(base + at * kv.page_stride, uint32_t(head_bytes));
      const int slot = ((st * kStep + 16 * u) & slot_mask) * kv.dim;
#pragma unroll
      for (int c = 0; c < DP / 64; ++c) {
        kreg[u][c] = u32x4{0, 0, 0, 0};
        if (!PAD || quarter * kQuarter + 16 * c < kv.dim)
          kreg[u][c] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, k_off + 16 * c, slot, 0);
      }
      const uint16_t* sc = kv.scale + at * kv.scale_stride + head;
      sk_bits[u] = __builtin_amdgcn_readfirstlane(sc[0]);
      sv_bits[u] = __builtin_amdgcn_readfirstlane(sc[kv.kv_heads]);
    }
  };
  auto load_v = [&](int st) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const long at = there(st, u) ? page[u] : 0;
      const auto rsrc = tile::make_rsrc(base + at * kv.page_stride + v_from, uint32_t(head_bytes));
      const int slot = ((st * kStep + 16 * u) & slot_mask) * kv.dim;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t (&w)[kVDwords] = vreg[4 * u + i];
        if (PAD) __builtin_memset(w, 0, sizeof(w));
        if (!PAD || r16 * kCols < kv.dim) {
          const int row_at = slot + i * kv.dim;
          if constexpr (kVDwords == 1) {
            w[0] = __builtin_amdgcn_raw_buffer_load_b32(rsrc, v_off, row_at, 0);
          } else if constexpr (kVDwords == 2) {
            const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(rsrc, v_off, row_at, 0);
            w[0] = x[0], w[1] = x[1];
          } else {
            const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(rsrc, v_off, row_at, 0);
            w[0] = x[0], w[1] = x[1], w[2] = x[2], w[3] = x[3];
          }
        }
      }
    }
  };

  f32x4 o[R][kCols];
  float m[R], l[R];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    m[j] = kNone;
    l[j] = 0.0f;
#pragma unroll
    for (int c = 0; c < kCols; ++c) o[j][c] = f32x4{0, 0, 0, 0};
  }

  int st = first + wave;
  if (st < last) {
    fetch_pages(st);
    load_k(st);
    load_v(st);
    fetch_pages(st + kWaves);
  }
  for (; st < last; st += kWaves) {
    // scores; the queries are read from LDS here, in every step
    f32x4 acc[R][2];
    int q_lane = lane;
    asm volatile("" : "+v"(q_lane));
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < kKStep; ++i) {
        const half8_t a = codes8(biased(kreg[u][i / 2][2 * (i % 2)]), biased(kreg[u][i / 2][2 * (i % 2) + 1]));
#pragma unroll
        for (int j = 0; j < R; ++j) {
          const f32x4 zero = {0, 0, 0, 0};
          half8_t qf;
          if constexpr (kHeld) qf = q[j][i];
          else qf = sh_q[j * kKStep + i][q_lane];
          acc[j][u] = mfma16(a, qf, i ? acc[j][u] : zero);
        }
        if (R > 1) __builtin_amdgcn_sched_barrier(0);
      }
    // factors of the step's two pages; a scale of 0 as in paged_attn.hip
    float sk[2], lv[2], rv[2];
    bool zero[2];
    const bool here[2] = {ok[0], ok[1]};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      sk[u] = key_scale(sk_bits[u]) * p.scale_log2e * kCodeScale;
      const float sv = h2f(uint16_t(sv_bits[u]));
      zero[u] = sv == 0.0f;
      const float sv1 = zero[u] ? 0x1p-24f : sv;
      lv[u] = __builtin_amdgcn_logf(sv1);
      rv[u] = __builtin_amdgcn_rcpf(sv1);
    }
    // the next step's keys, now that these are in the products
    if (st + kWaves < last) load_k(st + kWaves);

    // where some key is not seen by some row: scores with their scales here, minus
    // infinity for those, whatever their page's scale
    const int key0 = st * kStep;
    if (!(here[0] && here[1] && key0 + kStep <= min(start, range.hi) && key0 >= see_most)) {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        int t, q_head;
        const bool row_ok = row_of(j, &t, &q_head);
        const uint32_t bits = mask_window(p.mask + long(s.lo + t) * p.mask_ld, p.mask_words, key0 - start) >> 4 * quarter;
        const int key4 = key0 + 4 * quarter;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = key4 + 16 * u + i;
            const bool seen = row_ok && here[u] && (bits >> (16 * u + i) & 1) && key >= see_lo[j] && key < range.hi;
            acc[j][u][i] = seen ? __builtin_fmaf(acc[j][u][i], sk[u], lv[u]) : -__builtin_inff();
          }
      }
      sk[0] = sk[1] = 1.0f;
      lv[0] = lv[1] = 0.0f;
    }

    // weights of the rows: relative to the maximum they have, which moves only
    // when a weight would leave fp16's range
    half8_t pt[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      float sum[2];
      auto weights = [&](auto again) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          sum[u] = 0.0f;
          const float c = lv[u] - m[j];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // again: as the maximum was found, from the rounded score
            const float y = decltype(again)::value ? __builtin_fmaf(acc[j][u][i], sk[u], lv[u]) - m[j]
                                                   : __builtin_fmaf(acc[j][u][i], sk[u], c);
            const float e = __builtin_amdgcn_exp2f(y);
            sum[u] += e;
            pt[j][4 * u + i] = static_cast<_Float16>(e);
          }
        }
      };
      weights(std::false_type());
      if (__ballot(!(sum[0] + sum[1] <= kMost))) {
        float mx = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = fmaxf(mx, __builtin_fmaf(acc[j][i >> 2][i & 3], sk[i >> 2], lv[i >> 2]));
        const float m_new = fmaxf(m[j], lifted(row_max(mx)));
        const float alpha = __builtin_amdgcn_exp2f(m[j] - m_new);
        m[j] = m_new;
        l[j] *= alpha;
#pragma unroll
        for (int c = 0; c < kCols; ++c) o[j][c] *= alpha;
        weights(std::true_type());
      }
      // a sum of 0 (nothing seen) stays 0 whatever the page's scale holds
#pragma unroll
      for (int u = 0; u < 2; ++u) l[j] += sum[u] == 0.0f ? 0.0f : sum[u] * rv[u];
      if (R > 1) __builtin_amdgcn_sched_barrier(0);
    }
    // whatever the codes of a page with scale 0 are, its values are 0
    if (zero[0] || zero[1]) {
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) pt[j][i] = zero[i >> 2] ? (_Float16)0.0f : pt[j][i];
    }
    // values: 8 keys x kCols columns
#pragma unroll
    for (int c = 0; c < kVDwords; ++c) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = biased(vreg[i][c]);
#pragma unroll
      for (int col = 0; col < 4; ++col) {
        half8_t a;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const half2_t two = codes2(pair_bytes(w[i], w[i + 1], col));
          a[i] = two[0];
          a[i + 1] = two[1];
        }
#pragma unroll
        for (int j = 0; j < R; ++j) o[j][4 * c + col] = mfma16(a, pt[j], o[j][4 * c + col]);
        if (R > 1) __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (st + kWaves < last) {
      load_v(st + kWaves);
      fetch_pages(st + 2 * kWaves);
    }
  }

  // Join the four waves, a row tile at a time: lane holds result rows
  // 4 quarter + i, i.e. columns (4 quarter + i) * kCols + j of its row.
  __shared__ float sh_m[kWaves][16], sh_l[kWaves][16];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    l[j] = row_sum(l[j]);
    if (j || !kHeld) __syncthreads();
    if (quarter == 0) {
      sh_m[wave][r16] = m[j];
      sh_l[wave][r16] = l[j];
    }
#pragma unroll
    for (int c = 0; c < kCols; ++c) sh_o[wave][lane][c] = o[j][c];
    __syncthreads();
    int t, q_head;
    if (!row_of(j, &t, &q_head)) continue;
    float m_all = sh_m[0][r16];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m_all = fmaxf(m_all, sh_m[w][r16]);
    float l_all = 0.0f, factor[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      factor[w] = __builtin_amdgcn_exp2f(sh_m[w][r16] - m_all);
      l_all += sh_l[w][r16] * factor[w];
    }
    // wave w finishes result row i = w of each quarter: kCols columns
    const int d0 = (4 * quarter + wave) * kCols;
    if (PAD && d0 >= kv.dim) continue;
    float out[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += sh_o[w][lane][c][wave] * factor[w];
      out[c] = v;
    }
    if (p.splits == 1) {
      const float norm = l_all > 0.0f || l_all != l_all ? kCodeScale / l_all : 0.0f;
      uint16_t* dst = p.out + long(s.lo + t) * p.ldo + long(q_head) * kv.dim + d0;
#pragma unroll
      for (int c = 0; c < kCols; c += 4) {
        uint2 w;
        w.x = f2h_bits(out[c] * norm) | uint32_t(f2h_bits(out[c + 1] * norm)) << 16;
        w.y = f2h_bits(out[c + 2] * norm) | uint32_t(f2h_bits(out[c + 3] * norm)) << 16;
        *reinterpret_cast<uint2*>(dst + c) = w;
      }
    } else {
      const long at = (long(s.lo + t) * p.q_heads + q_head) * p.splits + split;
      if (quarter == 0 && wave == 0) p.part_ml[at] = make_float2(m_all, l_all);
      float4* dst = reinterpret_cast<float4*>(p.part_o + at * kv.dim + d0);
#pragma unroll
      for (int c = 0; c < kCols; c += 4) dst[c / 4] = make_float4(out[c], out[c + 1], out[c + 2], out[c + 3]);
    }
  }
}

template <int DP, bool PAD>
const void* kernel_of(int tiles) {
  if (tiles == 1) return reinterpret_cast<const void*>(&tree_attn_kernel<DP, PAD, 1>);
  if (tiles == 2) return reinterpret_cast<const void*>(&tree_attn_kernel<DP, PAD, 2>);
  if constexpr (DP <= 128) return reinterpret_cast<const void*>(&tree_attn_kernel<DP, PAD, 4>);
  return nullptr;                        // the plan takes at most two with heads above 128
}

}  // namespace

hipError_t launch_tree_attn(const AttnParams& p, int tiles, hipStream_t stream) {
  AttnParams a = p;
  void* args[] = {&a};
  const int dim = p.kv.dim;
  const long wgs = attn_tiles(p.kv, p.group, 16 * tiles) * p.kv.kv_heads * p.splits;
  const void* fn = dim == 64    ? kernel_of<64, false>(tiles)
                   : dim < 64   ? kernel_of<64, true>(tiles)
                   : dim == 128 ? kernel_of<128, false>(tiles)
                   : dim < 128  ? kernel_of<128, true>(tiles)
                   : dim == 256 ? kernel_of<256, false>(tiles)
                                : kernel_of<256, true>(tiles);
  return hipLaunchKernel(fn, dim3(unsigned(wgs)), dim3(kThreads), args, 0, stream);
}

}  // namespace w4a8
