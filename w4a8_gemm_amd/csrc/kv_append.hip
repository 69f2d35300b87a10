// Rotary positions on queries and keys, and keys and values appended to the
// paged int8 cache, in one launch (gfx950).
//
// A (page, k or v, kv head) of the cache is a block of page x dim codes under
// one fp16 scale.  New tokens may raise that scale: with s' = max(s, fp16(
// amax / 127)) the codes already there become rint(code * s / s'), which
// adds at most half a step of s' to them each time the scale grows.  One
// wave or workgroup owns a block for the whole call, so the scale, the old
// codes and the new ones change together without atomics.
//
// The first workgroups of the grid own blocks, the rest rotate queries.  Work
// items are 16 values: the two 8-value halves of 8 rotated pairs (positions j
// and j + rotary/2 in the half layout, 2j and 2j + 1 in the interleaved one),
// or 16 values that are not rotated.
//
// Measured: the next token of 64 sequences (32 + 8 heads of 128) 4.7 us, the
// latency of a launch and of loads that wait for each other (lengths, page number,
// the page's scale); 4 prompts of up to 1500 tokens (110 MB) 30 us = 3.7 TB/s
// into outputs that are not cached, 24.4 into the same ones, where a large copy
// reaches 5.2 TB/s.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "decoder_kernels.h"
#include "kv_page.h"
#include "quant_common.h"

namespace w4a8 {
namespace {

using namespace dev;

constexpr int kThreads = 256;

struct Item {
  int o1, o2;     // offsets of its two 8-value halves in the head
  int pair;       // first pair of its 8, or -1: not rotated
};

__device__ __forceinline__ Item item_of(int j, int rotary, bool interleaved) {
  Item it;
  const int half = rotary >> 1;
  if (j * 16 < rotary) {
    it.pair = j * 8;
    it.o1 = interleaved ? j * 16 : j * 8;
    it.o2 = interleaved ? j * 16 + 8 : half + j * 8;
  } else {
    it.pair = -1;
    it.o1 = j * 16;
    it.o2 = j * 16 + 8;
  }
  return it;
}

// an item as loaded: 16 fp16 values
struct Raw {
  uint4 a, b;
};

__device__ __forceinline__ Raw load_raw(const uint16_t* src, const Item& it) {
  return {*reinterpret_cast<const uint4*>(src + it.o1), *reinterpret_cast<const uint4*>(src + it.o2)};
}

__device__ __forceinline__ void unpack16(const Raw& r, float (&v)[16]) {
  uint16_t h[16];
  __builtin_memcpy(h, &r.a, 16);
  __builtin_memcpy(h + 8, &r.b, 16);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = h2f(h[i]);
}

struct Turn {
  float c[8], s[8];
};

__device__ __forceinline__ Turn turn_of(const AppendParams& p, const Item& it, int pos) {
  Turn t;
  const int half = p.rotary >> 1;
  const float* row = p.cos_sin + long(min(max(pos, 0), p.max_pos - 1)) * p.rotary + it.pair;
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    const float4 c = *reinterpret_cast<const float4*>(row + i);
    const float4 s = *reinterpret_cast<const float4*>(row + half + i);
    t.c[i] = c.x, t.c[i + 1] = c.y, t.c[i + 2] = c.z, t.c[i + 3] = c.w;
    t.s[i] = s.x, t.s[i + 1] = s.y, t.s[i + 2] = s.z, t.s[i + 3] = s.w;
  }
  return t;
}

// (a, b) -> (a cos - b sin, b cos + a sin) for the item's 8 pairs
__device__ __forceinline__ void rotate16(float (&v)[16], const Turn& t, bool interleaved) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int ia = interleaved ? 2 * i : i, ib = interleaved ? 2 * i + 1 : i + 8;
    const float a = v[ia], b = v[ib];
    v[ia] = a * t.c[i] - b * t.s[i];
    v[ib] = b * t.c[i] + a * t.s[i];
  }
}

// four fp32 values to int8 codes in one dword
__device__ __forceinline__ uint32_t codes4(const float* v, float r) {
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float y = __builtin_amdgcn_fmed3f(v[i] * r, -127.0f, 127.0f);
    b[i] = __builtin_bit_cast(uint32_t, y + 12582912.0f);
  }
  const uint32_t p01 = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
  const uint32_t p23 = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
  return p01 | p23;
}

// the dword's four codes under a scale `ratio` times as fine
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = float(int8_t(uint8_t(w >> (8 * i))));
  return codes4(v, ratio);
}

// WPB waves own a block (1: the block belongs to one wave, 4 blocks per
// workgroup; 4: to the workgroup).  Up to kHeld items a thread stay in
// registers from the search for their largest value to their quantization;
// larger blocks are read (and rotated) twice.
constexpr int kHeld = 2;

template <int WPB>
__device__ __forceinline__ void append_block(const AppendParams& p, int unit) {
  const KvArgs& kv = p.kv;
  constexpr int kTeam = WPB * 64;
  const int tid = WPB == 1 ? threadIdx.x & 63 : threadIdx.x;

  // unit -> (page slot, k or v, head); heads fastest: one token's heads lie
  // side by side in k and v
  const int head = unit % kv.kv_heads;
  const int which = (unit / kv.kv_heads) & 1;
  const int slot_index = unit / (2 * kv.kv_heads);
  int b, nth = 0;
  if (kv.cu_q) {
    b = kv::owner(slot_index, kv.batch,
                  [&](int i) { return (kv.cu_q[i] >> kv.page_shift) + 2 * i; }, &nth);
  } else {
    b = slot_index;
  }
  const kv::Seq s = kv::seq_of(kv, b);
  const int n = s.hi - s.lo;
  const int start = max(s.len - n, 0);                 // position of the first new token
  const int page_index = (start >> kv.page_shift) + nth;
  const int page_begin = page_index << kv.page_shift;
  const int begin = max(start, page_begin);            // new positions in this page
  const int end = min(s.len, page_begin + (1 << kv.page_shift));
  // every wave of a team takes the same way here
  if (nth < 0 || begin >= end) return;
  const int first = begin - page_begin;                // slots before it hold earlier tokens
  const int count = end - begin;
  const int token0 = s.hi - (s.len - begin);           // new token at position `begin`

  const uint16_t* src = (which ? p.v : p.k) + long(head) * kv.dim;
  const long ld = which ? p.ldv : p.ldk;
  const int rotary = which ? 0 : p.rotary;
  const bool inter = p.interleaved != 0;
  const int per_token = kv.dim >> 4;
  const int items = count * per_token;
  const bool held = items <= kHeld * kTeam;

  auto item = [&](int i, int* t) {
    *t = i / per_token;
    return item_of(i - *t * per_token, rotary, inter);
  };
  auto turn = [&](float (&v)[16], const Item& it, int t) {
    if (it.pair >= 0) rotate16(v, turn_of(p, it, begin + t), inter);
  };
  // the items' loads go out before the page's number and old scale are there
  Raw raw[kHeld];
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    const int i = tid + j * kTeam;
    int t;
    const Item it = item(i, &t);
    if (held && i < items) raw[j] = load_raw(src + (token0 + t) * ld, it);
  }
  const int page = kv::page_at(kv, b, page_index);
  if (page < 0) return;
  int8_t* block = kv.data + long(page) * kv.page_stride +
                  (long(which * kv.kv_heads + head) << kv.page_shift) * kv.dim;
  uint16_t* scale = kv.scale + long(page) * kv.scale_stride + which * kv.kv_heads + head;
  const uint32_t old_bits = first > 0 ? *scale & 0x7FFFu : 0u;

  float v[kHeld][16];
  uint32_t mx = 0;
  if (held) {
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int i = tid + j * kTeam;
      if (i >= items) continue;
      int t;
      const Item it = item(i, &t);
      unpack16(raw[j], v[j]);
      turn(v[j], it, t);
#pragma unroll
      for (int e = 0; e < 16; ++e) mx = max(mx, __builtin_bit_cast(uint32_t, v[j][e]) & 0x7FFFFFFFu);
    }
  } else {
    for (int i = tid; i < items; i += kTeam) {
      int t;
      const Item it = item(i, &t);
      unpack16(load_raw(src + (token0 + t) * ld, it), v[0]);
      turn(v[0], it, t);
#pragma unroll
      for (int e = 0; e < 16; ++e) mx = max(mx, __builtin_bit_cast(uint32_t, v[0][e]) & 0x7FFFFFFFu);
    }
  }
  mx = wave_max_u32(mx);
  if (WPB > 1) {
    __shared__ uint32_t wave_maxs[WPB];
    if ((threadIdx.x & 63) == 0) wave_maxs[threadIdx.x >> 6] = mx;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WPB; ++i) mx = max(mx, wave_maxs[i]);
  }
  const uint32_t new_bits = f2h_bits(__builtin_bit_cast(float, mx) / 127.0f);
  const uint32_t bits = max(old_bits, new_bits);       // fp16 patterns of values >= 0 (or NaN)
  const float r = act_recip(uint16_t(bits));
  // every thread has read the old scale: those of this wave before the
  // reduction, those of other waves before the barrier
  if (tid == 0) *scale = uint16_t(bits);

  if (first > 0 && bits != old_bits) {
    const float ratio = h2f(uint16_t(old_bits)) / h2f(uint16_t(bits));
    const int chunks = first * per_token;
    for (int i = tid; i < chunks; i += kTeam) {
      uint4* at = reinterpret_cast<uint4*>(block + long(i) * 16);
      uint4 w = *at;
      w.x = rescale4(w.x, ratio);
      w.y = rescale4(w.y, ratio);
      w.z = rescale4(w.z, ratio);
      w.w = rescale4(w.w, ratio);
      *at = w;
    }
  }
  auto store = [&](const float (&y)[16], const Item& it, int t) {
    int8_t* dst = block + (first + t) * kv.dim;
    *reinterpret_cast<uint2*>(dst + it.o1) = uint2{codes4(y, r), codes4(y + 4, r)};
    *reinterpret_cast<uint2*>(dst + it.o2) = uint2{codes4(y + 8, r), codes4(y + 12, r)};
  };
  if (held) {
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int i = tid + j * kTeam;
      if (i >= items) continue;
      int t;
      const Item it = item(i, &t);
      store(v[j], it, t);
    }
  } else {
    for (int i = tid; i < items; i += kTeam) {
      int t;
      const Item it = item(i, &t);
      unpack16(load_raw(src + (token0 + t) * ld, it), v[0]);
      turn(v[0], it, t);
      store(v[0], it, t);
    }
  }
}

// Queries: one item of one token, HEADS heads of it (the cosines stay in
// registers).
template <int HEADS>
__device__ __forceinline__ void rotate_queries(const AppendParams& p, long index) {
  const KvArgs& kv = p.kv;
  const int per_token = kv.dim >> 4;
  const int parts = (p.q_heads + HEADS - 1) / HEADS;
  const int j = int(index % per_token);
  const long rest = index / per_token;
  const int part = int(rest % parts);
  const long t = rest / parts;
  if (t >= kv.total_q) return;
  const bool inter = p.interleaved != 0;
  const Item it = item_of(j, p.rotary, inter);
  const int h0 = part * HEADS;
  Raw raw[HEADS];
#pragma unroll
  for (int h = 0; h < HEADS; ++h)
    if (h0 + h < p.q_heads) raw[h] = load_raw(p.q + t * p.ldq + long(h0 + h) * kv.dim, it);
  Turn turn;
  if (it.pair >= 0) {
    int b = int(t), nth = 0;
    if (kv.cu_q) b = kv::owner(int(t), kv.batch, [&](int i) { return kv.cu_q[i]; }, &nth);
    const kv::Seq s = kv::seq_of(kv, b);
    turn = turn_of(p, it, s.len - s.hi + int(t));
  }
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    if (h0 + h >= p.q_heads) continue;
    float v[16];
    unpack16(raw[h], v);
    if (it.pair >= 0) rotate16(v, turn, inter);
    uint16_t o[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = f2h_bits(v[e]);
    uint4 a, b4;
    __builtin_memcpy(&a, o, 16);
    __builtin_memcpy(&b4, o + 8, 16);
    uint16_t* dst = p.q_out + t * p.ldqo + long(h0 + h) * kv.dim;
    *reinterpret_cast<uint4*>(dst + it.o1) = a;
    *reinterpret_cast<uint4*>(dst + it.o2) = b4;
  }
}

template <int WPB, int HEADS>
__global__ __launch_bounds__(kThreads) void rope_append_kernel(AppendParams p, int block_wgs,
                                                               int units) {
  if (int(blockIdx.x) < block_wgs) {
    const int unit = WPB == 1 ? int(blockIdx.x) * 4 + (threadIdx.x >> 6) : int(blockIdx.x);
    if (unit < units) append_block<WPB>(p, unit);
    return;
  }
  rotate_queries<HEADS>(p, long(blockIdx.x - block_wgs) * kThreads + threadIdx.x);
}

}  // namespace

hipError_t launch_rope_append(const AppendParams& p, hipStream_t stream) {
  const bool small = append_small(p.kv);
  const long block_wgs = append_block_wgs(p.kv);
  const long wgs = block_wgs + append_query_wgs(p.kv, p.q_heads);
  AppendParams a = p;
  int bw = int(block_wgs), un = int(append_slots(p.kv) * 2 * p.kv.kv_heads);
  void* args[] = {&a, &bw, &un};
  const void* fn = small ? reinterpret_cast<const void*>(&rope_append_kernel<1, 1>)
                         : reinterpret_cast<const void*>(&rope_append_kernel<4, 4>);
  return hipLaunchKernel(fn, dim3(unsigned(wgs)), dim3(kThreads), args, 0, stream);
}

}  // namespace w4a8
