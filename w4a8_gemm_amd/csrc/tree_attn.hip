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
// The waves join through LDS.  Where row tiles do not fill the device, each is
// split over its keys, so that about as many equal parts come out as workgroups
// can run at once, and tree_join_kernel joins them.
//
// Bound by vector instructions: of a wave's step with 32 rows (about 300, 1400
// cycles, where its 32 matrix instructions take 512) half convert codes and half
// are the softmax.  A small batch is bound by latency: loads that wait for each
// other, and code that runs once and has to be fetched, about a nanosecond a byte.
// Measured, graph replays with the join: 16 trees of up to 64 tokens over up to
// 4096 keys, heads 32 / 8 of 128, 73 us = 0.32 PFLOP/s; 4 of up to 13 over 50000
// 71 us = 3.4 TB/s; 6 of up to 200 over 1700 under a window of 1024, heads 16 / 4
// of 64, 20 us; one of 26 over 2001 13.8 us.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attn_common.h"
#include "kv_page.h"
#include "quant_common.h"
#include "verify_kernels.h"

namespace w4a8 {
namespace {

using namespace attn;
using namespace dev;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = kTreeStep;   // keys a wave takes at once
// A lane's weights of a step may add up to this (fp16 ends at 65504).
constexpr float kMost = 65000.0f;

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// over the four lanes of a row (lane, lane ^ 16, lane ^ 32, ...)
__device__ __forceinline__ float row_max(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const float y = fmaxf(__builtin_bit_cast(float, uint32_t(a[0])), __builtin_bit_cast(float, uint32_t(a[1])));
  const uint32_t v = __builtin_bit_cast(uint32_t, y);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return fmaxf(__builtin_bit_cast(float, uint32_t(b[0])), __builtin_bit_cast(float, uint32_t(b[1])));
}
__device__ __forceinline__ float row_sum(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const float y = __builtin_bit_cast(float, uint32_t(a[0])) + __builtin_bit_cast(float, uint32_t(a[1]));
  const uint32_t v = __builtin_bit_cast(uint32_t, y);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return __builtin_bit_cast(float, uint32_t(b[0])) + __builtin_bit_cast(float, uint32_t(b[1]));
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

// A sequence's work for one kv head: its row tiles, each of the same steps.
struct Work {
  int b;
  kv::Seq s;
  int n, start;               // drafted tokens, position of the first
  int all_lo;                 // no row sees keys before
  int tiles, first, steps;    // first: the step that holds all_lo
};

template <int ROWS>
__device__ __forceinline__ Work work_of(const TreeAttnParams& p, int b) {
  Work w;
  w.b = b;
  w.s = kv::seq_of(p.kv, b);
  w.n = w.s.hi - w.s.lo;
  w.start = w.s.len - w.n;
  w.all_lo = p.window > 0 ? max(w.start - p.window, 0) : 0;
  w.tiles = (w.n * p.group + ROWS - 1) / ROWS;
  w.first = w.all_lo / kStep;
  w.steps = max((w.s.len + kStep - 1) / kStep - w.first, 1);
  return w;
}

// the same of one sequence for all lanes, as scalars
template <int ROWS>
__device__ __forceinline__ Work wave_work_of(const TreeAttnParams& p, int b) {
  Work w = work_of<ROWS>(p, b);
  w.s.lo = __builtin_amdgcn_readfirstlane(w.s.lo);
  w.n = __builtin_amdgcn_readfirstlane(w.n);
  w.s.hi = w.s.lo + w.n;
  w.s.len = __builtin_amdgcn_readfirstlane(w.s.len);
  w.start = w.s.len - w.n;
  w.all_lo = __builtin_amdgcn_readfirstlane(w.all_lo);
  w.tiles = __builtin_amdgcn_readfirstlane(w.tiles);
  w.first = __builtin_amdgcn_readfirstlane(w.first);
  w.steps = __builtin_amdgcn_readfirstlane(w.steps);
  return w;
}

// Sums of the lanes up to each: within rows of 16, then the rows before.
__device__ __forceinline__ int wave_upto(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);    // from 1, 2, 4, 8 lanes below
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);    // row 0's last to row 1, 2's to 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);    // the first half's to the second
  return x;
}

// A workgroup's part of a row tile.
struct Part {
  Work w;
  int tile, parts, nth;       // of the tile's parts the nth: the steps
  int first, last;            // [first, last) of the sequence
};

__device__ __forceinline__ int parts_of(const Work& w, int share) {
  return share > 0 ? (w.steps + share - 1) / share : 1;
}

// The parts of all sequences in a line, sequence after sequence, tile after tile,
// and the `mine`th of them; false where there are fewer.  A sequence's tiles are
// split into equal parts of at most `share` steps, so that about p.shares parts
// come out in all; 0 shares: not split.  The lanes of a wave look through as many
// sequences each; all take part.  A lane counts no more than kMostWork, which a
// proper cu_q does not reach (work is counted in units of 2^p.unit steps), so that
// an improper one makes no sum overflow.
template <int ROWS>
__device__ __forceinline__ bool part_of(const TreeAttnParams& p, int mine, int lane, Part* part) {
  const int batch = p.kv.batch, each = (batch + 63) >> 6;
  int share = 0, from = 0, b = 0;
  if (p.shares > 0) {
    int work = 0, tiles = 0;
    for (int i = 0; i < each; ++i) {
      if (lane * each + i < batch) {
        const Work w = work_of<ROWS>(p, lane * each + i);
        work = int(min(work + long(w.tiles) * ((w.steps >> p.unit) + 1), kMostWork));
        tiles = int(min(long(tiles) + w.tiles, kMostWork));
      }
    }
    work = __builtin_amdgcn_readlane(wave_upto(work), 63);
    tiles = __builtin_amdgcn_readlane(wave_upto(tiles), 63);
    const int room = max(p.shares - tiles, 1);
    share = int(min(max((long(work) + room - 1) / room << p.unit, long(p.least)), kMostWork));
  }
  if (batch > kTreeBatch) {               // not split: a search, each tile's place from cu_q alone
    int unused;
    if (p.kv.cu_q) {
      auto first = [&](int i) { return int(long(p.kv.cu_q[i]) * p.group / ROWS) + i; };
      b = kv::owner(mine, batch, first, &unused);
      from = first(b);
    } else {
      const int per = (p.group + ROWS - 1) / ROWS;
      b = mine / per;
      from = b * per;
    }
  } else {
    // the lane with the part's sequence, then the sequence among that lane's
    for (int turn = 0; turn < 2; ++turn) {
      const int count = turn ? 1 : each;
      int here = 0;
      if (turn == 0 || lane < each) {
        for (int i = 0; i < count; ++i) {
          const int at = turn ? b + lane : lane * each + i;
          if (at < batch) {
            const Work w = work_of<ROWS>(p, at);
            here = int(min(here + long(w.tiles) * parts_of(w, share), kMostWork));
          }
        }
      }
      const int upto = wave_upto(here);
      const uint64_t beyond = __ballot(upto > mine - from);
      if (!beyond) return false;
      const int l = __builtin_ctzll(beyond);
      if (l > 0) from += __builtin_amdgcn_readlane(upto, l - 1);
      b = turn ? b + l : l * each;
      if (each == 1) break;
    }
  }
  b = __builtin_amdgcn_readfirstlane(min(b, batch - 1));
  part->w = wave_work_of<ROWS>(p, b);
  part->parts = __builtin_amdgcn_readfirstlane(parts_of(part->w, share));
  const int in = mine - __builtin_amdgcn_readfirstlane(from);
  part->tile = __builtin_amdgcn_readfirstlane(in / part->parts);
  part->nth = in - part->tile * part->parts;
  // equal parts, whole turns of the waves
  const int size = (part->w.steps + part->parts * kWaves - 1) / (part->parts * kWaves) * kWaves;
  part->first = __builtin_amdgcn_readfirstlane(min(part->nth * size, part->w.steps)) + part->w.first;
  part->last = __builtin_amdgcn_readfirstlane(min((part->nth + 1) * size, part->w.steps)) + part->w.first;
  return part->tile >= 0 && part->tile < part->w.tiles;
}

// DP: head dim rounded up to 64, 128 or 256.  PAD: dim < DP.  P16: pages of 16
// keys, so that the two halves of a step lie in two.  R: row tiles of 16 that a
// workgroup takes; the queries of one tile of up to 128 values or two of 64 stay in
// registers, others are read from LDS at each step.
template <int DP, bool PAD, bool P16, int R>
__global__ __launch_bounds__(kThreads, DP * R > 256 ? 2 : 3) void tree_attn_kernel(TreeAttnParams p) {
  constexpr int kRows = 16 * R;
  constexpr int kQuarter = DP / 4;        // K bytes of a lane and key
  constexpr int kKStep = DP / 32;         // products of one 16-key score tile
  constexpr int kCols = DP / 16;          // V columns of a lane
  constexpr int kVDwords = DP / 64;       // dwords of those columns and one key
  constexpr bool kHeld = DP * R <= 128;
  constexpr bool kLate = DP * R > 256;
  const KvArgs& kv = p.kv;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int r16 = lane & 15, quarter = lane >> 4;

  // LDS: what the rows see, and the waves' results at the end, before that the
  // queries where they are not held
  __shared__ float sh_m[kWaves][16], sh_l[kWaves][16];
  __shared__ int2 sh_row[64];             // drafted token (-1: no row), first position seen
  __shared__ f32x4 sh_o[kWaves][64][kCols + 1];
  static_assert(R * kKStep * 64 * sizeof(half8_t) <= sizeof(sh_o), "the queries fit");
  half8_t (*const sh_q)[64] = reinterpret_cast<half8_t (*)[64]>(&sh_o[0][0][0]);

  // Heads fastest: neighbouring workgroups go to different dies, so that a die
  // keeps few heads' keys in its L2.
  const int head = blockIdx.x % kv.kv_heads;
  Part part;
  if (!part_of<kRows>(p, blockIdx.x / kv.kv_heads, lane, &part)) return;     // the whole workgroup
  const Work& work = part.w;
  const kv::Seq s = work.s;
  const int n = work.n, rows = n * p.group, start = work.start, nth = part.tile;
  const int first = part.first, last = part.last;
  const int hi = min(last * kStep, s.len);                  // keys before it are this workgroup's

  // A row of the tile: drafted token and query head.  The tile's first row is
  // divided by the group once; the few further rows through a multiplication
  // (exact while rows times group fit 32 bits).
  const int t0 = nth * kRows / p.group, rest0 = nth * kRows - t0 * p.group;
  const int left = rows - 1 - nth * kRows;                  // its last row
  auto row_of = [&](int row, int* t, int* q_head) {
    const int r = rest0 + min(row, left);
    const int step = p.group == 1 ? r : int(__umulhi(uint32_t(r), p.group_inverse));
    *t = t0 + step;
    *q_head = head * p.group + r - step * p.group;
    return row <= left;
  };
  // What rows see is worked out a lane each
  int see_most = 0;                                         // no row's window begins later
  {
    int t, unused, see_lo = 0;
    const bool ok = row_of(lane, &t, &unused) && lane < kRows;
    if (p.window > 0) {
      see_lo = window_begin(p.mask + long(s.lo + t) * p.mask_ld, p.mask_words, n, start, p.window);
      see_most = __builtin_amdgcn_readfirstlane(wave_max_u32(ok ? see_lo : 0));
    }
    if (wave == 0) sh_row[lane] = make_int2(ok ? t : -1, see_lo);
  }

  // Q^T fragments: lane's row, d = quarter * DP/4 + 8 i ..
  half8_t q[kHeld ? R : 1][kHeld ? kKStep : 1];
  auto load_q = [&](int j, half8_t (&to)[kKStep]) {
    int t, q_head;
    const bool ok = row_of(16 * j + r16, &t, &q_head);
    const uint16_t* src = p.q + long(s.lo + t) * p.ldq + long(q_head) * kv.dim;
#pragma unroll
    for (int i = 0; i < kKStep; ++i) {
      const int d = quarter * kQuarter + 8 * i;
      uint4 u = {0, 0, 0, 0};
      if (ok && (!PAD || d < kv.dim)) u = *reinterpret_cast<const uint4*>(src + d);
      to[i] = query8(__builtin_bit_cast(half8_t, u));
    }
  };
  if constexpr (kHeld) {
#pragma unroll
    for (int j = 0; j < R; ++j) load_q(j, q[j]);
  } else {
    for (int j = wave; j < R; j += kWaves) {
      half8_t now[kKStep];
      load_q(j, now);
#pragma unroll
      for (int i = 0; i < kKStep; ++i) sh_q[j * kKStep + i][lane] = now[i];
    }
  }
  __syncthreads();

  // Loads: the 16 keys of a half step lie in one page, as do all 32 where pages
  // hold more, so addresses are scalar up to the lane's fixed offset.
  constexpr int kPages = P16 ? 2 : 1;     // of a step
  constexpr int kPageKeys = kStep / kPages;
  const int dim = PAD ? kv.dim : DP;
  const long head_bytes = long(dim) << kv.page_shift;
  const int8_t* const base = kv.data + head * head_bytes;
  const long v_from = kv.kv_heads * head_bytes;
  const int32_t* const table = kv.table + long(work.b) * kv.table_ld;
  const int slot_mask = (1 << kv.page_shift) - 1;
  const unsigned k_off = unsigned(r16 * dim + quarter * kQuarter);
  const unsigned v_off = unsigned(quarter * 4 * dim + r16 * kCols);
  int page[kPages];
  auto fetch_pages = [&](int st) {
#pragma unroll
    for (int u = 0; u < kPages; ++u) {
      const int key = min(st * kStep + kPageKeys * u, hi - 1);
      page[u] = kv::scalar_load(table + (max(key, 0) >> kv.page_shift));
    }
  };
  u32x4 kreg[2][DP / 64];
  uint32_t vreg[8][kVDwords];
  uint32_t scales[kPages];                // even lanes: of keys, odd ones: of values
  bool ok[kPages];
  const int8_t* at_keys[kPages];          // of the step whose keys were asked for last
  auto load_k = [&](int st) {
#pragma unroll
    for (int u = 0; u < kPages; ++u) {
      const int key = st * kStep + kPageKeys * u;
      ok[u] = key < hi && page[u] >= 0 && page[u] < kv.num_pages;
      const long at = ok[u] ? page[u] : 0;      // page 0 where there is none
      const int8_t* from = base + at * kv.page_stride + (key & slot_mask) * dim;
      at_keys[u] = from;
#pragma unroll
      for (int half = P16 ? u : 0; half < (P16 ? u + 1 : 2); ++half)
#pragma unroll
        for (int c = 0; c < DP / 64; ++c) {
          kreg[half][c] = u32x4{0, 0, 0, 0};
          if (!PAD || quarter * kQuarter + 16 * c < dim)
            kreg[half][c] = *reinterpret_cast<const u32x4*>(from + (P16 ? 0 : 16 * half * dim) + 16 * c + k_off);
        }
      scales[u] = kv.scale[at * kv.scale_stride + head + (lane & 1) * kv.kv_heads];
    }
  };
  auto load_v = [&]() {                   // of the same step
#pragma unroll
    for (int u = 0; u < kPages; ++u) {
      const int8_t* from = at_keys[u] + v_from;
#pragma unroll
      for (int half = P16 ? u : 0; half < (P16 ? u + 1 : 2); ++half)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t (&w)[kVDwords] = vreg[4 * half + i];
          if (PAD) __builtin_memset(w, 0, sizeof(w));
          if (!PAD || r16 * kCols < dim)
            __builtin_memcpy(w, __builtin_assume_aligned(from + ((P16 ? 0 : 16 * half) + i) * dim + v_off, kCols), kCols);
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
    if (!kLate) load_v();
    fetch_pages(st + kWaves);
  }
  for (; st < last; st += kWaves) {
    // scores; queries that are not held are read from LDS here, a product ahead
    f32x4 acc[R][2];
    half8_t ahead[2][R];
    int q_lane = lane;
    asm volatile("" : "+v"(q_lane));
    auto read_q = [&](int i) {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if constexpr (kHeld) ahead[i & 1][j] = q[j][i];
        else ahead[i & 1][j] = sh_q[j * kKStep + i][q_lane];
      }
    };
    read_q(0);
#pragma unroll
    for (int i = 0; i < kKStep; ++i) {
      if (i + 1 < kKStep) read_q(i + 1);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const half8_t a = codes8(biased(kreg[u][i / 2][2 * (i % 2)]), biased(kreg[u][i / 2][2 * (i % 2) + 1]));
#pragma unroll
        for (int j = 0; j < R; ++j) {
          const f32x4 zero = {0, 0, 0, 0};
          acc[j][u] = mfma16(a, ahead[i & 1][j], i ? acc[j][u] : zero);
        }
      }
    }
    // factors of the step's two pages; a scale of 0 as in paged_attn.hip
    float sk[kPages], lv[kPages], rv[kPages];
    bool zero[kPages], here[kPages], all_here = true, any_zero = false;
#pragma unroll
    for (int u = 0; u < kPages; ++u) {
      here[u] = ok[u];
      all_here &= ok[u];
      sk[u] = key_scale(__builtin_amdgcn_readlane(scales[u], 0)) * p.scale_log2e * kCodeScale;
      const float sv = h2f(uint16_t(__builtin_amdgcn_readlane(scales[u], 1)));
      zero[u] = sv == 0.0f;
      any_zero |= zero[u];
      const float sv1 = zero[u] ? 0x1p-24f : sv;
      lv[u] = __builtin_amdgcn_logf(sv1);
      rv[u] = __builtin_amdgcn_rcpf(sv1);
    }
    // Keys and values are asked for as early as registers allow: values as soon as
    // the step before is done with its own and keys as soon as these are in the
    // products, or, with 32 rows of long heads, a stretch before they are used.
    if (kLate) load_v();
    else if (st + kWaves < last) load_k(st + kWaves);

    // where some key is not seen by some row: scores with their scales here, minus
    // infinity for those, whatever their page's scale
    const int key0 = st * kStep;
    if (!(all_here && key0 + kStep <= min(start, hi) && key0 >= see_most)) {
      // the step's keys that the lane's row sees, a bit each
      uint32_t seen = 0;
      const int2 row = sh_row[lane];
      if (row.x >= 0) seen = mask_window(p.mask + long(s.lo + row.x) * p.mask_ld, p.mask_words, key0 - start);
      if (row.y > key0) seen = row.y - key0 < 32 ? seen & ~0u << (row.y - key0) : 0u;
      if (hi - key0 < 32) seen &= (1u << max(hi - key0, 0)) - 1;
      if (P16) seen &= (here[0] ? 0xFFFFu : 0u) | (here[kPages - 1] ? 0xFFFF0000u : 0u);
      else if (!here[0]) seen = 0;
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const uint32_t bits = uint32_t(__builtin_amdgcn_ds_bpermute(4 * r16 + 64 * j, int(seen))) >> 4 * quarter;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = __builtin_fmaf(acc[j][u][i], sk[P16 ? u : 0], lv[P16 ? u : 0]);
            acc[j][u][i] = bits >> (16 * u + i) & 1 ? x : -__builtin_inff();
          }
      }
#pragma unroll
      for (int u = 0; u < kPages; ++u) {
        sk[u] = 1.0f;
        lv[u] = 0.0f;
      }
    }

    // weights of the rows: relative to the maximum they have, which moves only
    // when a weight would leave fp16's range
    half8_t pt[R];
    float sum[R][kPages];
    auto weights = [&](int j, auto again) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int u = P16 ? half : 0;
        if (P16 || half == 0) sum[j][u] = 0.0f;
        const float c = lv[u] - m[j];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // again: as the maximum was found, from the rounded score
          const float y = decltype(again)::value ? __builtin_fmaf(acc[j][half][i], sk[u], lv[u]) - m[j]
                                                 : __builtin_fmaf(acc[j][half][i], sk[u], c);
          const float e = __builtin_amdgcn_exp2f(y);
          sum[j][u] += e;
          pt[j][4 * half + i] = static_cast<_Float16>(e);
        }
      }
    };
    auto most = [&](int j) { return P16 ? sum[j][0] + sum[j][kPages - 1] : sum[j][0]; };
    bool fits = true;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      weights(j, std::false_type());
      fits &= most(j) <= kMost;
    }
    if (__ballot(!fits)) {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if (!__ballot(!(most(j) <= kMost))) continue;
        float mx = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int u = P16 ? i >> 2 : 0;
          mx = fmaxf(mx, __builtin_fmaf(acc[j][i >> 2][i & 3], sk[u], lv[u]));
        }
        const float m_new = fmaxf(m[j], lifted(row_max(mx)));
        const float alpha = __builtin_amdgcn_exp2f(m[j] - m_new);
        m[j] = m_new;
        l[j] *= alpha;
#pragma unroll
        for (int c = 0; c < kCols; ++c) o[j][c] *= alpha;
        weights(j, std::true_type());
      }
    }
    // a sum of 0 (nothing seen) stays 0 whatever the page's scale holds
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int u = 0; u < kPages; ++u) l[j] += sum[j][u] == 0.0f ? 0.0f : sum[j][u] * rv[u];
    if (kLate && st + kWaves < last) load_k(st + kWaves);
    // whatever the codes of a page with scale 0 are, its values are 0
    if (any_zero) {
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) pt[j][i] = zero[P16 ? i >> 2 : 0] ? (_Float16)0.0f : pt[j][i];
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
      }
    }
    if (st + kWaves < last) {
      if (!kLate) load_v();
      fetch_pages(st + 2 * kWaves);
    }
  }

  // Join the four waves, a row tile at a time: lane holds result rows
  // 4 quarter + i, i.e. columns (4 quarter + i) * kCols + j of its row.
  const bool whole = part.parts == 1;
#pragma unroll 1
  for (int j = 0; j < R; ++j) {
    if (j || !kHeld) __syncthreads();
#pragma unroll
    for (int x = 0; x < R; ++x) {
      if (j != x) continue;
      const float sum = row_sum(l[x]);
      if (quarter == 0) {
        sh_m[wave][r16] = m[x];
        sh_l[wave][r16] = sum;
      }
#pragma unroll
      for (int c = 0; c < kCols; ++c) sh_o[wave][lane][c] = o[x][c];
    }
    __syncthreads();
    int t, q_head;
    const bool row_ok = row_of(16 * j + r16, &t, &q_head);
    float m_all = sh_m[0][r16];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m_all = fmaxf(m_all, sh_m[w][r16]);
    float l_all = 0.0f, factor[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      factor[w] = __builtin_amdgcn_exp2f(sh_m[w][r16] - m_all);
      l_all += sh_l[w][r16] * factor[w];
    }
    // wave w finishes columns w * kMine .. of each of the lane's four result rows
    // (16-byte reads at an odd stride: no two lanes of eight share a bank)
    constexpr int kMine = kCols / kWaves;
    f32x4 out[kMine];
#pragma unroll
    for (int c = 0; c < kMine; ++c) {
      out[c] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) out[c] += sh_o[w][lane][wave * kMine + c] * factor[w];
    }
    const float norm = l_all > 0.0f || l_all != l_all ? kCodeScale / l_all : 0.0f;
    const long to = long(blockIdx.x) * kRows + 16 * j + r16;     // of a part's row
    if (!whole && row_ok && quarter == 0 && wave == 0) p.part_ml[to] = make_float2(m_all, l_all);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d0 = (4 * quarter + i) * kCols + wave * kMine;
      if (!row_ok || (PAD && d0 >= kv.dim)) continue;
      if (whole) {
        uint16_t h[kMine];
#pragma unroll
        for (int c = 0; c < kMine; ++c) h[c] = f2h_bits(out[c][i] * norm);
        __builtin_memcpy(p.out + long(s.lo + t) * p.ldo + long(q_head) * kv.dim + d0, h, 2 * kMine);
      } else {
        float x[kMine];
#pragma unroll
        for (int c = 0; c < kMine; ++c) x[c] = out[c][i];
        __builtin_memcpy(__builtin_assume_aligned(p.part_o + to * kv.dim + d0, 4 * kMine), x, 4 * kMine);
      }
    }
  }
}

// Row tiles in several parts.  The workgroups that had a part, but the first,
// divide the tile's rows.
template <int ROWS>
__global__ __launch_bounds__(256) void tree_join_kernel(TreeAttnParams p) {
  const KvArgs& kv = p.kv;
  const int head = blockIdx.x % kv.kv_heads;
  Part part;
  if (!part_of<ROWS>(p, blockIdx.x / kv.kv_heads, threadIdx.x & 63, &part) || part.nth == 0) return;
  const int parts = part.parts;
  const int rows = min(part.w.n * p.group - part.tile * ROWS, ROWS);
  const long slot0 = (long(blockIdx.x) - long(part.nth) * kv.kv_heads) * ROWS;   // of the first part's rows
  const long slot_step = long(kv.kv_heads) * ROWS;
  const int per = kv.dim >> 2;                      // lanes of a row
  const int groups = 256 / per;
  const int lane = threadIdx.x % per, group = threadIdx.x / per;
  // few parts: a row belongs to one group; else all groups share a row's parts,
  // with two barriers a row.  Up to 4, 8, 16 and 32 parts measured, us: 4 trees of 13
  // tokens over 50000 keys 75, 73, 71 and 71; 3 of them 71, 72, 69 and 68.
  const bool shared = parts > 16;
  __shared__ float4 sh_o[256];
  __shared__ float2 sh_ml[256];
  const int stride = (parts - 1) * (shared ? 1 : groups);
  for (int base = (part.nth - 1) * (shared ? 1 : groups); base < rows; base += stride) {
    const int row = base + (shared ? 0 : group);
    float m = kNone, l = 0.0f;
    float4 o = {0, 0, 0, 0};
    auto add = [&](float2 a, float4 v) {
      const float top = fmaxf(m, a.x);
      const float f = __builtin_amdgcn_exp2f(m - top), e = __builtin_amdgcn_exp2f(a.x - top);
      m = top;
      l = l * f + a.y * e;
      o.x = o.x * f + v.x * e;
      o.y = o.y * f + v.y * e;
      o.z = o.z * f + v.z * e;
      o.w = o.w * f + v.w * e;
    };
    if (group < groups && row < rows) {
#pragma unroll 4
      for (int i = shared ? group : 0; i < parts; i += shared ? groups : 1) {
        const long at = slot0 + i * slot_step + row;
        add(p.part_ml[at], *reinterpret_cast<const float4*>(p.part_o + at * kv.dim + 4 * lane));
      }
    }
    if (shared) {
      __syncthreads();                              // the row before has been read
      sh_o[threadIdx.x] = o;
      sh_ml[threadIdx.x] = make_float2(m, l);
      __syncthreads();
      if (group > 0) continue;
      for (int i = 1; i < groups; ++i) add(sh_ml[i * per + lane], sh_o[i * per + lane]);
    }
    if (group >= groups || row >= rows) continue;
    const int r = part.tile * ROWS + row, t = r / p.group, q_head = head * p.group + r - t * p.group;
    const float norm = l > 0.0f || l != l ? kCodeScale / l : 0.0f;
    uint2 w;
    w.x = f2h_bits(o.x * norm) | uint32_t(f2h_bits(o.y * norm)) << 16;
    w.y = f2h_bits(o.z * norm) | uint32_t(f2h_bits(o.w * norm)) << 16;
    *reinterpret_cast<uint2*>(p.out + long(part.w.s.lo + t) * p.ldo + long(q_head) * kv.dim + 4 * lane) = w;
  }
}

template <int DP, bool PAD, bool P16>
const void* kernel_of(int tiles) {
  if (tiles == 1)
    return reinterpret_cast<const void*>(&tree_attn_kernel<DP, PAD, P16, 1>);
  return reinterpret_cast<const void*>(&tree_attn_kernel<DP, PAD, P16, 2>);
}
template <bool P16>
const void* kernel_of(int dim, int tiles) {
  return dim == 64    ? kernel_of<64, false, P16>(tiles)
         : dim < 64   ? kernel_of<64, true, P16>(tiles)
         : dim == 128 ? kernel_of<128, false, P16>(tiles)
         : dim < 128  ? kernel_of<128, true, P16>(tiles)
         : dim == 256 ? kernel_of<256, false, P16>(tiles)
                      : kernel_of<256, true, P16>(tiles);
}

}  // namespace

hipError_t launch_tree_attn(const TreeAttnParams& p, hipStream_t stream) {
  TreeAttnParams a = p;
  void* args[] = {&a};
  const long wgs = long(p.groups) * p.kv.kv_heads;
  const void* fn = p.kv.page_shift == 4 ? kernel_of<true>(p.kv.dim, p.tiles) : kernel_of<false>(p.kv.dim, p.tiles);
  const hipError_t e = hipLaunchKernel(fn, dim3(unsigned(wgs)), dim3(kThreads), args, 0, stream);
  if (e != hipSuccess || p.shares == 0) return e;
  fn = p.tiles == 1 ? reinterpret_cast<const void*>(&tree_join_kernel<16>)
                    : reinterpret_cast<const void*>(&tree_join_kernel<32>);
  return hipLaunchKernel(fn, dim3(unsigned(wgs)), dim3(256), args, 0, stream);
}

}  // namespace w4a8
