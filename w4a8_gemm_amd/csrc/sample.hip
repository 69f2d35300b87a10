// Tokens drawn from rows of logits (gfx950): temperature, top-k, top-p, min-p and
// one given random number a row.
//
// A token's weight is exp((x - max) / T), held as a whole number of 2^-44: sums
// of such numbers are exact in any order, so that what is drawn does not depend
// on how a row is split, and 2^-44 of the largest weight is far below what a
// random number of 24 bits can tell apart.
//
// The tokens that the filters keep are the first ones in the order of falling
// logits (equal ones by number): all above some logit, and the first few that
// have it.  That logit is found from its leading bits on, by counting tokens
// (top-k) or adding their weights (top-p) in bins of those bits.  Then each wave
// adds up the kept weights of its stretches of the row, and the stretch that
// holds the drawn token is looked through.
//
// Long rows are read by many workgroups first.
//   sample_max_kernel    the largest logit of every 128 bytes.  The top_k-th largest
//                        of these bounds the tokens that may be kept: few, and in
//                        few groups, so that the row is not read again.
//   sample_sum_kernel    where all weights count, their sums: by stretches, or for
//                        top_p in 2048 bins of 1/32 of log2 weight
//   sample_split_kernel  for top_p, the bin in which its share is reached: weights
//                        above it by stretches, and the bin's tokens as a list
//
// Reading bounds sample_max_kernel (244 MB 48 us, 5 TB/s).  Where all weights count,
// their powers of two in 64 bits bound sample_sum_kernel and sample_split_kernel,
// about 30 instructions a logit; in bins, also the additions in LDS.  sample_kernel
// is latency: two dozen barriers, 7 to 14 us, and two rows a compute unit.
// Measured, graph replays of the whole call: one row of 32000 fp16 logits with top_k
// and top_p 16.5 us (21 in one kernel); 64 of 128256 with top_p 50 (max
// 7, sums 17, split 15, drawing 13); 801 of 152064, settings of each row's own, 211
// (48, 47, 44, 71); 33 of 50257 fp32 with min_p 10.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "quant_common.h"
#include "verify_kernels.h"

namespace w4a8 {
namespace {

using namespace dev;

// Two workgroups of 512 fit a compute unit, one of 1024.  1024 measured, us: 801 rows of
// 152064 with top_k 50 134 against 109, with top_p 341 and 314, one row with top_k 50
// 23.7 and 26.5 (19.6 since groups are found first).
constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kBinBits = 11;
constexpr int kBins = 1 << kBinBits;
constexpr int kParts = kBins + 64;       // stretches of 64 chunks in a row of W4A8_VOCAB_MAX logits
constexpr int kUnitBits = 44;            // weights count units of 2^-44
static_assert(W4A8_VOCAB_MAX <= 1 << 19, "a row's weights add up in 63 bits, its stretches fit kParts");

// 2^f on [-1/2, 1/2]: the polynomial through 11 Chebyshev points, off by 2^-51
__device__ __forceinline__ double exp2_near0(double f) {
  double r = 7.072585949269223e-09;
  r = __builtin_fma(r, f, 1.0208690299958306e-07);
  r = __builtin_fma(r, f, 1.321544258792169e-06);
  r = __builtin_fma(r, f, 1.5252657260200837e-05);
  r = __builtin_fma(r, f, 0.0001540353044173605);
  r = __builtin_fma(r, f, 0.0013333558230164974);
  r = __builtin_fma(r, f, 0.009618129107606888);
  r = __builtin_fma(r, f, 0.05550410866444772);
  r = __builtin_fma(r, f, 0.24022650695910097);
  r = __builtin_fma(r, f, 0.69314718055995);
  return __builtin_fma(r, f, 1.0);
}

// Logits as ordered keys: a larger logit has a larger key, equal ones the same
// (-0 is 0).  kLowest is minus infinity's.
template <typename T>
struct Logit;
template <>
struct Logit<uint16_t> {
  static constexpr int kBits = 16, kEach = 8;
  static constexpr uint32_t kLowest = 0x03FF, kNone = 0xFC00;
  static __device__ __forceinline__ uint32_t key(uint32_t b) {
    b = b == 0x8000u ? 0u : b;
    return b & 0x8000u ? ~b & 0xFFFFu : b | 0x8000u;
  }
  static __device__ __forceinline__ uint32_t key_of(float v) { return key(f2h_bits(v)); }
  static __device__ __forceinline__ double of_bits(uint32_t b) { return double(h2f(uint16_t(b))); }
  static __device__ __forceinline__ double value(uint32_t key) {
    return double(h2f(uint16_t(key & 0x8000u ? key ^ 0x8000u : ~key)));
  }
  static __device__ __forceinline__ bool bad(uint32_t b) { return (b & 0x7FFFu) >= 0x7C00u && b != 0xFC00u; }
};
template <>
struct Logit<uint32_t> {
  static constexpr int kBits = 32, kEach = 4;
  static constexpr uint32_t kLowest = 0x007FFFFF, kNone = 0xFF800000;
  static __device__ __forceinline__ uint32_t key(uint32_t b) {
    b = b == 0x80000000u ? 0u : b;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
  }
  static __device__ __forceinline__ uint32_t key_of(float v) { return key(__builtin_bit_cast(uint32_t, v)); }
  static __device__ __forceinline__ double of_bits(uint32_t b) { return double(__builtin_bit_cast(float, b)); }
  static __device__ __forceinline__ double value(uint32_t key) {
    return double(__builtin_bit_cast(float, key & 0x80000000u ? key ^ 0x80000000u : ~key));
  }
  static __device__ __forceinline__ bool bad(uint32_t b) {
    return (b & 0x7FFFFFFFu) >= 0x7F800000u && b != 0xFF800000u;
  }
};

// A row in chunks of 16 aligned bytes; the first and the last may hold less.
template <typename T>
struct Row {
  static constexpr int kEach = Logit<T>::kEach;
  const T* from;              // the aligned bytes that hold the first logit
  int head, end;              // its place there, and the place behind the last
  int chunks;
  // chunk c as it lies in memory, minus infinity where there is no logit
  __device__ __forceinline__ uint4 load(int c) const {
    const int at = c * kEach;
    if (at >= head && at + kEach <= end) return *reinterpret_cast<const uint4*>(from + at);
    T raw[kEach];
    for (int e = 0; e < kEach; ++e)
      raw[e] = at + e >= head && at + e < end ? from[at + e] : T(Logit<T>::kNone);
    uint4 v;
    __builtin_memcpy(&v, raw, 16);
    return v;
  }
  // f(chunk, its four dwords) for all chunks of the row; the lanes of a wave get
  // neighbouring chunks, all waves take part equally often
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    for (int base = 0; base < chunks; base += kThreads) {
      const int c = base + int(threadIdx.x);
      const uint4 v = load(c);
      const uint32_t mine[4] = {v.x, v.y, v.z, v.w};
      f(c, mine);
    }
  }
};

// logit e of a chunk, as its bits
template <typename T>
__device__ __forceinline__ uint32_t bits_of(const uint32_t (&w)[4], int e) {
  return sizeof(T) == 4 ? w[e & 3] : w[(e >> 1) & 3] >> 16 * (e & 1) & 0xFFFFu;
}

constexpr int kList = kSampleList;
// Up to so many listed tokens are ranked by looking at all for each, n^2 / 64 steps of
// a wave: 256 take about 10 us, what a selection among more and the sums of
// stretches take.
constexpr int kFew = 256;

struct Shared {
  uint64_t mass[kParts];      // of bins, then of stretches
  uint32_t count[kParts];
  uint64_t sums[kWaves];
  uint64_t found_before;
  int found;
  uint2 list[kList];          // (key, place) of the tokens that may be kept, in no order
  int listed;                 // their number; more than kList: not listed
  uint4 few[kFew];            // (weight's two words, place, key) of kept tokens
  int fews, hits;
};

// Sums of the lanes up to each: within rows of 16, then the rows before.
template <int CONTROL, int ROWS>
__device__ __forceinline__ uint64_t lanes_before(uint64_t x) {
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, uint32_t(x), CONTROL, ROWS, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, uint32_t(x >> 32), CONTROL, ROWS, 0xF, false);
  return lo | uint64_t(hi) << 32;
}
__device__ __forceinline__ uint64_t wave_upto(uint64_t x) {
  x += lanes_before<0x111, 0xF>(x);              // from 1, 2, 4, 8 lanes below
  x += lanes_before<0x112, 0xF>(x);
  x += lanes_before<0x114, 0xF>(x);
  x += lanes_before<0x118, 0xF>(x);
  x += lanes_before<0x142, 0xA>(x);              // row 0's last to row 1, 2's to 3
  return x + lanes_before<0x143, 0xC>(x);        // the first half's to the second
}
__device__ __forceinline__ uint64_t last_lane(uint64_t x) {
  return uint32_t(__builtin_amdgcn_readlane(uint32_t(x), 63)) |
         uint64_t(uint32_t(__builtin_amdgcn_readlane(uint32_t(x >> 32), 63))) << 32;
}

// Sums of the threads before this one; *total that of all.  All threads call it.
template <int THREADS = kThreads, typename S>
__device__ __forceinline__ uint64_t block_before(S& sh, uint64_t x, uint64_t* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint64_t upto = wave_upto(x);
  __syncthreads();                        // the last call's sums have been read
  if (lane == 63) sh.sums[wave] = upto;
  __syncthreads();
  uint64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    if (w < wave) before += sh.sums[w];
    all += sh.sums[w];
  }
  *total = all;
  return before + upto - x;
}

// The first i of n for which the values up to it reach the target, and the sum
// before it; -1 if their total does not.  The target (1 or more) is given for
// the total.  All threads call it and get the same.
template <int THREADS = kThreads, typename S, typename Value, typename Target>
__device__ __forceinline__ int find(S& sh, int n, Value value, Target target_of, uint64_t* before,
                                    uint64_t* target, uint64_t* total) {
  const int per = (n + THREADS - 1) / THREADS;
  const int from = min(int(threadIdx.x) * per, n), to = min(from + per, n);
  uint64_t mine = 0;
  for (int i = from; i < to; ++i) mine += value(i);
  if (threadIdx.x == 0) sh.found = -1;
  uint64_t at = block_before<THREADS>(sh, mine, total);
  *target = target_of(*total);
  if (at < *target && *target <= at + mine) {
    for (int i = from; i < to; ++i) {
      const uint64_t v = value(i);
      if (*target <= at + v) {
        sh.found = i;
        sh.found_before = at;
        break;
      }
      at += v;
    }
  }
  __syncthreads();
  *before = sh.found_before;
  return sh.found;
}

// The settings of a row, and its largest logit.
struct Settings {
  float temperature, top_p, min_p;
  int top_k;
};
__device__ __forceinline__ Settings settings_of(const SampleParams& p, long r) {
  Settings s;
  s.temperature = p.s.temperature_dev ? p.s.temperature_dev[r] : p.s.temperature;
  s.top_k = p.s.top_k_dev ? p.s.top_k_dev[r] : p.s.top_k;
  s.top_p = p.s.top_p_dev ? p.s.top_p_dev[r] : p.s.top_p;
  s.min_p = p.s.min_p_dev ? p.s.min_p_dev[r] : p.s.min_p;
  if (s.top_k >= p.vocab) s.top_k = 0;
  return s;
}
__device__ __forceinline__ bool valid(const Settings& s) {
  return s.temperature >= 0.0f && s.temperature != __builtin_inff() && s.top_p == s.top_p && s.min_p == s.min_p;
}
// whether the weights of all the row's tokens count, and whether in bins
__device__ __forceinline__ bool in_bins(const Settings& s) {
  return s.temperature > 0.0f && s.top_k <= 0 && s.top_p < 1.0f;
}
__device__ __forceinline__ bool sums_all(const Settings& s) {
  return s.temperature > 0.0f && s.top_k <= 0 && s.top_p >= 1.0f && s.min_p <= 0.0f;
}
// how much of a row's weight top_p asks for
__device__ __forceinline__ uint64_t share_of(const Settings& s, uint64_t all) {
  const double want = __builtin_ceil(double(fmaxf(s.top_p, 0.0f)) * double(all));
  return max(uint64_t(want), uint64_t(1));
}
// the least weight that min_p keeps, in units of 2^-44
__device__ __forceinline__ double least_of(const Settings& s) {
  return double(s.min_p > 0.0f ? fminf(s.min_p, 1.0f) : 0.0f) * (1ull << kUnitBits);
}

template <typename T>
__device__ __forceinline__ Row<T> row_of(const SampleParams& p, long r) {
  Row<T> row;
  const T* at = static_cast<const T*>(p.logits) + r * p.ld;
  row.head = int((reinterpret_cast<uintptr_t>(at) & 15u) / sizeof(T));
  row.from = at - row.head;
  row.end = row.head + p.vocab;
  row.chunks = (row.end + Row<T>::kEach - 1) / Row<T>::kEach;
  return row;
}

// weights of a row, as multiples of 2^-44 before and after rounding
template <typename T>
struct Weigh {
  double largest, turn;
  __device__ __forceinline__ Weigh(uint32_t top, float temperature)
      : largest(Logit<T>::value(top)), turn(1.4426950408889634 / double(temperature)) {}
  // log2 of the weight
  __device__ __forceinline__ double log2_of(uint32_t key) const { return (Logit<T>::value(key) - largest) * turn; }
  __device__ __forceinline__ double log2_of_bits(uint32_t bits) const { return (Logit<T>::of_bits(bits) - largest) * turn; }
  __device__ __forceinline__ double operator()(uint32_t key) const { return of_log2(log2_of(key)); }
  // 2^(t + 44): adding 1.5 * 2^52 rounds t to a whole number, which stands in the
  // sum's low bits and is added to the exponent of 2^(the rest)
  static __device__ __forceinline__ double of_log2(double t) {
    const double sum = t + 0x1.8p52;
    const int whole = int(__builtin_bit_cast(uint64_t, sum));
    const uint64_t w = __builtin_bit_cast(uint64_t, exp2_near0(t - (sum - 0x1.8p52)));
    const double y = __builtin_bit_cast(double, w + (uint64_t(uint32_t(whole + kUnitBits) << 20) << 32));
    return t > -64.0 ? y : 0.0;
  }
};
__device__ __forceinline__ uint64_t units(double w) {
  return __builtin_bit_cast(uint64_t, w + 0x1p52) & ((1ull << 52) - 1);
}

__device__ __forceinline__ uint64_t wave_sum64(uint64_t x) { return last_lane(wave_upto(x)); }

// What long rows are asked before: workgroups of 256 threads take kSpan chunks.
constexpr int kAheadThreads = 256;
constexpr int kSpan = kSampleSpan;
constexpr int kLoads = kSpan / kAheadThreads;
constexpr int kGroup = kSampleGroup;     // chunks of a group: neighbouring lanes

template <typename T>
__global__ __launch_bounds__(kAheadThreads) void sample_max_kernel(SampleParams p) {
  using L = Logit<T>;
  const int block = blockIdx.x % p.blocks;
  const long r = blockIdx.x / p.blocks;
  const Row<T> row = row_of<T>(p, r);
  const int groups = p.groups;
  if (p.bins) {
    for (int i = block * kAheadThreads + int(threadIdx.x); i < kSampleBins; i += p.blocks * kAheadThreads)
      p.bins[r * kSampleBins + i] = 0;
    if (block == 0 && threadIdx.x == 0) p.listed[r] = 0;
  }
  uint4 v[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) v[i] = row.load(block * kSpan + i * kAheadThreads + int(threadIdx.x));
  uint32_t top = L::kLowest;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint32_t most = L::kLowest;
#pragma unroll
    for (int e = 0; e < L::kEach; ++e) {
      const uint32_t b = bits_of<T>(w, e);
      bad |= L::bad(b);
      most = max(most, L::key(b));
    }
    top = max(top, most);
    // over the eight lanes of a group
    most = max(most, uint32_t(__builtin_amdgcn_update_dpp(0u, most, 0x141, 0xF, 0xF, false)));
    most = max(most, uint32_t(__builtin_amdgcn_update_dpp(0u, most, 0x4E, 0xF, 0xF, false)));
    most = max(most, uint32_t(__builtin_amdgcn_update_dpp(0u, most, 0xB1, 0xF, 0xF, false)));
    const int group = (block * kSpan + i * kAheadThreads + int(threadIdx.x)) / kGroup;
    if (threadIdx.x % kGroup == 0 && group < groups) p.maxima[r * groups + group] = most;
  }
  top = wave_max_u32(top);
  __shared__ uint32_t tops[kAheadThreads / 64];
  __shared__ int bads[kAheadThreads / 64];
  const bool any = __ballot(bad) != 0;
  if ((threadIdx.x & 63) == 0) {
    tops[threadIdx.x >> 6] = top;
    bads[threadIdx.x >> 6] = any;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    uint64_t all = top | uint64_t(any) << 32;
#pragma unroll
    for (int w = 1; w < kAheadThreads / 64; ++w) all = max(uint32_t(all), tops[w]) | (all >> 32 | bads[w]) << 32;
    p.tops[r * p.blocks + block] = all;
  }
}

// What the kernels after the first share: the row's largest logit and this
// workgroup's chunks.
template <typename T>
__device__ __forceinline__ uint32_t top_of(const SampleParams& p, long r, int lane) {
  uint32_t top = Logit<T>::kLowest;
  for (int i = lane; i < p.blocks; i += 64) top = max(top, uint32_t(p.tops[r * p.blocks + i]));
  return wave_max_u32(top);
}
template <typename T>
__device__ __forceinline__ void load_span(const Row<T>& row, int block, uint32_t (&w)[4 * kLoads]) {
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const uint4 v = row.load(block * kSpan + i * kAheadThreads + int(threadIdx.x));
    w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
  }
}
// The bin of a weight: larger ones first, all of one weight in one.
__device__ __forceinline__ int bin_of(double log2_weight) {
  return int(fmin(log2_weight * -32.0, double(kSampleBins - 1)));
}

template <typename T>
__global__ __launch_bounds__(kAheadThreads) void sample_sum_kernel(SampleParams p) {
  using L = Logit<T>;
  const int block = blockIdx.x % p.blocks;
  const long r = blockIdx.x / p.blocks;
  const Settings s = settings_of(p, r);
  const bool bins = in_bins(s);
  if (!valid(s) || !(bins || sums_all(s))) return;
  const int lane = threadIdx.x & 63;
  uint32_t w[4 * kLoads];
  load_span(row_of<T>(p, r), block, w);
  const Weigh<T> weight(top_of<T>(p, r, lane), s.temperature);
  __shared__ unsigned long long sums[kSampleBins];
  if (bins) {
    for (int i = threadIdx.x; i < kSampleBins; i += kAheadThreads) sums[i] = 0;
    __syncthreads();
  }
#pragma unroll 1
  for (int i = 0; i < kLoads; ++i) {
    const uint32_t mine[4] = {w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
    uint64_t mass = 0;
#pragma unroll
    for (int e = 0; e < L::kEach; ++e) {
      // minus infinity, also where there is no logit, weighs 0
      const double t = weight.log2_of_bits(bits_of<T>(mine, e));
      const uint64_t x = units(weight.of_log2(t));
      if (bins) {
        if (x) atomicAdd(&sums[bin_of(t)], static_cast<unsigned long long>(x));
      } else {
        mass += x;
      }
    }
    if (bins) continue;
    mass = wave_sum64(mass);
    const int part = (block * kSpan + i * kAheadThreads + int(threadIdx.x)) >> 6;
    if (lane == 0 && part < p.parts) p.masses[r * p.parts + part] = mass;
  }
  if (!bins) return;
  __syncthreads();
  for (int i = threadIdx.x; i < kSampleBins; i += kAheadThreads)
    if (sums[i]) atomicAdd(reinterpret_cast<unsigned long long*>(&p.bins[r * kSampleBins + i]), sums[i]);
}

struct SplitShared {
  uint64_t sums[kAheadThreads / 64];
  uint64_t found_before;
  int found;
  int listed, from;
  uint2 list[kSpan];
};

template <typename T>
__global__ __launch_bounds__(kAheadThreads) void sample_split_kernel(SampleParams p) {
  using L = Logit<T>;
  __shared__ SplitShared sh;
  const int block = blockIdx.x % p.blocks;
  const long r = blockIdx.x / p.blocks;
  const Settings s = settings_of(p, r);
  if (!valid(s) || !in_bins(s)) return;
  const int lane = threadIdx.x & 63;
  uint32_t w[4 * kLoads];
  load_span(row_of<T>(p, r), block, w);
  const uint32_t top = top_of<T>(p, r, lane);
  if (threadIdx.x == 0) sh.listed = 0;
  uint64_t before, target, total;
  const uint64_t* const bins = p.bins + r * kSampleBins;
  const int bin = find<kAheadThreads>(sh, kSampleBins, [&](int i) { return bins[i]; },
                                      [&](uint64_t all) { return share_of(s, all); }, &before, &target, &total);
  if (bin < 0) return;                          // nothing to draw from
  const Weigh<T> weight(top, s.temperature);
  const double least = least_of(s);
#pragma unroll 1
  for (int i = 0; i < kLoads; ++i) {
    const uint32_t mine[4] = {w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
    const int c = block * kSpan + i * kAheadThreads + int(threadIdx.x);
    uint64_t mass = 0;
#pragma unroll
    for (int e = 0; e < L::kEach; ++e) {
      const uint32_t bits = bits_of<T>(mine, e);
      const double t = weight.log2_of_bits(bits);
      const int in = t > -64.0 ? bin_of(t) : kSampleBins;
      if (in < bin) {
        const double x = weight.of_log2(t);
        if (x >= least) mass += units(x);
      } else if (in == bin) {
        const int at = atomicAdd(&sh.listed, 1);
        if (at < kSpan) sh.list[at] = make_uint2(L::key(bits), c * L::kEach + e);
      }
    }
    mass = wave_sum64(mass);
    const int part = c >> 6;
    if (lane == 0 && part < p.parts) p.masses[r * p.parts + part] = mass;
  }
  __syncthreads();
  // this workgroup's place in the row's list; too many, here or in all, make it not
  // a list
  if (threadIdx.x == 0 && sh.listed)
    sh.from = atomicAdd(&p.listed[r], sh.listed > kSpan ? kSampleList + 1 : sh.listed);
  __syncthreads();
  const int n = min(sh.listed, kSpan);
  for (int i = threadIdx.x; i < n && sh.from + i < kSampleList; i += kAheadThreads)
    p.list[r * kSampleList + sh.from + i] = sh.list[i];
}

template <typename T>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleParams p) {
  using L = Logit<T>;
  constexpr int kEach = L::kEach;
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const long r = blockIdx.x;
  const Row<T> row = row_of<T>(p, r);
  const Settings s = settings_of(p, r);
  const float u_raw = p.u[r];
  const bool ahead = p.maxima != nullptr;       // the two kernels before have run
  const uint32_t* const maxima = p.maxima + r * p.groups;

  auto finish = [&](int place, float prob) {
    p.tokens[r] = place - row.head;
    if (p.probs) p.probs[r] = prob;
  };

  // the largest logit, of each thread and of the row, and its first place
  bool bad = !valid(s);
  uint32_t mine = L::kLowest, mine_at = 0;
  if (ahead) {
    for (int i = tid; i < p.blocks; i += kThreads) {
      const uint64_t x = p.tops[r * p.blocks + i];
      mine = max(mine, uint32_t(x));
      bad |= x >> 32 != 0;
    }
  } else {
    row.each([&](int c, const uint32_t (&w)[4]) {
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const uint32_t b = bits_of<T>(w, e), key = L::key(b);
        bad |= L::bad(b);
        if (key > mine) {
          mine = key;
          mine_at = c * kEach + e;
        }
      }
    });
  }
  uint32_t top = wave_max_u32(mine);
  const bool wave_bad = __ballot(bad) != 0;
  if (lane == 0) sh.sums[wave] = top | uint64_t(wave_bad) << 32;
  if (tid == 0) sh.listed = sh.fews = sh.hits = 0;
  __syncthreads();
  bad = false;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    top = max(top, uint32_t(sh.sums[w]));
    bad |= sh.sums[w] >> 32 != 0;
  }
  if (bad || top == L::kLowest) {
    if (tid == 0) finish(row.head - 1, bad ? __builtin_nanf("") : 0.0f);
    return;
  }
  if (s.temperature == 0.0f || s.top_k == 1) {
    // a thread's first place with its largest is the first of all it has
    if (ahead) {
      mine = L::kLowest;
      for (int g = tid; g < p.groups && mine != top; g += kThreads) {
        mine = maxima[g];
        mine_at = g;
      }
    }
    uint32_t first = wave_max_u32(mine == top ? ~mine_at : 0u);
    __syncthreads();
    if (lane == 0) sh.sums[wave] = first;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) first = max(first, uint32_t(sh.sums[w]));
    if (!ahead) {
      if (tid == 0) finish(int(~first), 1.0f);
      return;
    }
    // the place in its group
    uint32_t place = ~0u;
    if (tid < kGroup) {
      const uint4 v = row.load(int(~first) * kGroup + tid);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = kEach - 1; e >= 0; --e)
        if (L::key(bits_of<T>(w, e)) == top) place = (int(~first) * kGroup + tid) * kEach + e;
    }
    if (wave == 0) {
      place = ~wave_max_u32(~place);
      if (tid == 0) finish(int(place), 1.0f);
    }
    return;
  }

  const Weigh<T> weight(top, s.temperature);
  const double least = least_of(s);
  const float u = u_raw >= 0.0f ? fminf(u_raw, 0x1.fffffep-1f) : 0.0f;
  auto target_of = [&](uint64_t all) { return uint64_t(double(u) * double(all)) + 1; };

  // The tokens kept: keys above `border`, and the first `ties` that have it.  Once
  // they are known to lie among few, these are in sh.list.
  uint32_t border = L::kLowest;
  uint64_t ties = 0;
  bool listed = false;
  auto each_listed = [&](auto f) {
    for (int i = tid; i < sh.listed; i += kThreads) f(sh.list[i].x, sh.list[i].y);
  };
  auto add_to_list = [&](uint32_t key, uint32_t place) {
    if (*const_cast<volatile int*>(&sh.listed) > kList) return;      // too many: not a list
    const int at = atomicAdd(&sh.listed, 1);
    if (at < kList) sh.list[at] = make_uint2(key, place);
  };
  // all tokens with keys of at least `from`, if they fit
  auto gather = [&](uint32_t from) {
    auto look = [&](int c, const uint32_t (&w)[4]) {
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const uint32_t key = L::key(bits_of<T>(w, e));
        if (key >= from) add_to_list(key, c * kEach + e);
      }
    };
    if (ahead) {
      // the groups that have such tokens first: each has at least one
      int* const hits = reinterpret_cast<int*>(sh.mass);
      for (int g = tid; g < p.groups; g += kThreads) {
        if (maxima[g] < from) continue;
        const int at = atomicAdd(&sh.hits, 1);
        if (at < kList) hits[at] = g;
      }
      __syncthreads();
      const int n = sh.hits;
      if (n > kList) return;                     // listed stays false
      for (int i = tid / kGroup; i < n; i += kThreads / kGroup) {
        const int c = hits[i] * kGroup + tid % kGroup;
        const uint4 v = row.load(c);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        look(c, w);
      }
    } else {
      row.each(look);
    }
    __syncthreads();
    listed = sh.listed <= kList;
  };
  // Finds the key at which counts (MASS: weights) of tokens, added from the largest
  // key down, reach the target; what is left of the target there.  The tokens are
  // those kept so far, from the row or the list; MAXIMA: the largest of the groups,
  // or of the threads.
  auto select = [&](auto mass_tag, auto maxima_tag, auto target_of, uint32_t* key_out, uint64_t* left) {
    constexpr bool kMass = decltype(mass_tag)::value, kMaxima = decltype(maxima_tag)::value;
    uint32_t prefix = 0;
    uint64_t target = 0;
    const uint64_t border_mass = kMass && ties ? ties * units(weight(border)) : 0;
#pragma unroll 1
    for (int shift = L::kBits; shift > 0;) {
      const int width = min(kBinBits, shift), low = shift - width;
      const bool first = shift == L::kBits;
      __syncthreads();
      for (int i = tid; i < kBins; i += kThreads) {
        if (kMass) sh.mass[i] = 0;
        else sh.count[i] = 0;
      }
      __syncthreads();
      auto add = [&](uint32_t key) {
        if (key <= border || !(first || key >> (shift & 31) == prefix)) return;
        const uint32_t bin = key >> low & ((1u << width) - 1);
        if constexpr (kMass) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.mass[bin]), units(weight(key)));
        else atomicAdd(&sh.count[bin], 1u);
      };
      if constexpr (kMaxima) {
        if (ahead) {
          for (int g = tid; g < p.groups; g += kThreads) add(maxima[g]);
        } else {
          add(mine);
        }
      } else if (listed) {
        each_listed([&](uint32_t key, uint32_t) { add(key); });
      } else {
        row.each([&](int c, const uint32_t (&w)[4]) {
#pragma unroll
          for (int e = 0; e < kEach; ++e) add(L::key(bits_of<T>(w, e)));
        });
      }
      if (kMass && tid == 0 && border_mass && (first || border >> (shift & 31) == prefix))
        atomicAdd(reinterpret_cast<unsigned long long*>(&sh.mass[border >> low & ((1u << width) - 1)]), border_mass);
      __syncthreads();
      const int n = 1 << width;
      uint64_t before, total;
      const int at = find(sh, n, [&](int i) { return kMass ? sh.mass[n - 1 - i] : uint64_t(sh.count[n - 1 - i]); },
                          [&](uint64_t all) { return first ? target_of(all) : target; }, &before, &target, &total);
      if (at < 0) return false;
      target -= before;
      prefix = prefix << width | uint32_t(n - 1 - at);
      shift = low;
      // of maxima only a bound is wanted
      if (kMaxima && shift <= 10) {
        *key_out = max(prefix << shift, L::kLowest + 1);
        return true;
      }
      // what is kept has at least these leading bits
      if (!kMaxima && !listed && shift > 0) {
        __syncthreads();
        if (tid == 0) sh.listed = sh.hits = 0;
        __syncthreads();
        gather(max(prefix << shift, ties ? border : border + 1));
      }
    }
    *key_out = prefix;
    *left = target;
    return true;
  };
  // Draws from the listed tokens, all there are that may be kept, a thread each: a
  // token's place in the order of falling logits, and the weights before it there
  // and in the order of numbers, are worked out by looking at all.
  auto from_few = [&](int most) {
    const int n = sh.listed;
    uint2 own = {0, 0};
    uint64_t mass = 0;
    double w = 0.0;
    if (tid < n) {
      own = sh.list[tid];
      w = weight(own.x);
      mass = units(w);
      sh.few[tid] = make_uint4(uint32_t(mass), uint32_t(mass >> 32), own.y, own.x);
    }
    __syncthreads();
    int rank = 0;
    uint64_t before = 0;
    if (tid < n) {
      for (int i = 0; i < n; ++i) {
        const uint4 x = sh.few[i];
        const bool first = x.w > own.x || (x.w == own.x && x.z < own.y);
        rank += first;
        before += first ? x.x | uint64_t(x.y) << 32 : 0;
      }
      if (rank == min(most, n) - 1) sh.found_before = before + mass;      // of all that count
    }
    __syncthreads();
    if (tid < n) {
      const bool kept = rank < most && (s.top_p >= 1.0f || before < share_of(s, sh.found_before)) && w >= least;
      if (!kept) mass = 0;
      sh.few[tid].x = uint32_t(mass);
      sh.few[tid].y = uint32_t(mass >> 32);
    }
    __syncthreads();
    if (tid >= n || mass == 0) return;
    uint64_t upto = 0, all = 0;
    for (int i = 0; i < n; ++i) {
      const uint4 x = sh.few[i];
      const uint64_t m = x.x | uint64_t(x.y) << 32;
      all += m;
      upto += x.z <= own.y ? m : 0;
    }
    const uint64_t target = target_of(all);
    if (upto >= target && upto - mass < target) finish(int(own.y), float(w / double(all)));
  };
  // The n-th largest of the maxima is not above the n-th largest of all logits.  It
  // bounds well where n is small beside their number, and not at all beyond it: one
  // row of 32000 normal fp16 logits (500 groups) with top_k 50 16.6 us, 256 45, 400 71,
  // 499 203, 501 58, 1000 96, 2048 222.
  const bool by_count = s.top_k > 0, by_mass = s.top_p < 1.0f;
  uint32_t at_key;
  uint64_t left;
  if (by_count && s.top_k <= (ahead ? kList : kThreads) / 2) {
    if (select(std::false_type(), std::true_type(), [&](uint64_t) { return uint64_t(s.top_k); }, &at_key, &left))
      gather(at_key);
    if (listed && sh.listed <= kFew) {
      from_few(s.top_k);
      return;
    }
  } else if (ahead && !by_count && !by_mass && least > 0.0) {
    // only min_p: a logit that is certainly not above the least one kept
    // (its weight as computed; the largest temperatures round many to 1)
    const double down = (log(double(fminf(s.min_p, 1.0f))) - 1e-12) * double(s.temperature);
    const double from = weight.largest + down - 1e-12 * (fabs(weight.largest) - down);
    gather(max(L::key_of(float(from)) - 1, L::kLowest + 1));
    if (listed && sh.listed <= kFew) {
      from_few(kFew);
      return;
    }
  }
  if (by_count &&
      select(std::false_type(), std::false_type(), [&](uint64_t) { return uint64_t(s.top_k); }, &at_key, &left)) {
    border = at_key;
    ties = left;
  }
  bool split = false;                   // the list holds one bin; weights above it are in p.masses
  if (by_mass) {
    auto part_of = [&](uint64_t all) { return share_of(s, all); };
    uint64_t target = 0;
    if (ahead && in_bins(s) && p.listed[r] <= kList) {
      const uint64_t* const bins = p.bins + r * kSampleBins;
      uint64_t before, total;
      __syncthreads();
      split = find(sh, kSampleBins, [&](int i) { return bins[i]; }, part_of, &before, &target, &total) >= 0;
      target -= before;
      if (tid == 0) sh.listed = p.listed[r];
      for (int i = tid; i < p.listed[r]; i += kThreads) sh.list[i] = p.list[r * kSampleList + i];
      listed = split;
      __syncthreads();
    }
    if (select(std::true_type(), std::false_type(), [&](uint64_t all) { return split ? target : part_of(all); }, &at_key, &left)) {
      const uint64_t each = units(weight(at_key));
      border = at_key;
      ties = (left + each - 1) / each;
    }
  }
  const double border_weight = weight(border);
  const uint64_t border_units = units(border_weight);
  if (border == L::kLowest || border_weight < least) ties = 0;
  auto kept = [&](uint32_t key, double* w) -> uint64_t {
    if (key <= border) return 0;
    *w = weight(key);
    return *w >= least ? units(*w) : 0;
  };

  if (listed && !split) {
    // From few tokens: each one's place among them is worked out by looking at all.
    __syncthreads();
    each_listed([&](uint32_t key, uint32_t place) {
      double w = border_weight;
      uint64_t mass = kept(key, &w);
      if (key == border && ties) {
        uint64_t rank = 0;
        for (int i = 0; i < sh.listed; ++i) rank += sh.list[i].x == border && sh.list[i].y < place;
        if (rank < ties) mass = border_units;
      }
      if (mass) {
        const int at = atomicAdd(&sh.fews, 1);
        if (at < kFew) sh.few[at] = make_uint4(uint32_t(mass), uint32_t(mass >> 32), place, key);
      }
    });
    __syncthreads();
    const int n = sh.fews;
    if (n <= kFew) {
      if (tid >= n) return;
      const uint4 own = sh.few[tid];
      uint64_t upto = 0, all = 0;
      for (int i = 0; i < n; ++i) {
        const uint4 x = sh.few[i];
        const uint64_t mass = x.x | uint64_t(x.y) << 32;
        all += mass;
        upto += x.z <= own.z ? mass : 0;
      }
      const uint64_t target = target_of(all);
      if (upto >= target && upto - (own.x | uint64_t(own.y) << 32) < target)
        finish(int(own.z), float(weight(own.w) / double(all)));
      return;
    }
  }

  // kept weight of every stretch of 64 chunks, without and then with the tokens
  // at the border
  const int parts = (row.chunks + 63) / 64;
  __syncthreads();
  if (listed || (ahead && sums_all(s))) {
    for (int i = tid; i < parts; i += kThreads) {
      sh.mass[i] = listed && !split ? 0 : p.masses[r * p.parts + i];
      sh.count[i] = 0;
    }
    if (listed) {
      __syncthreads();
      each_listed([&](uint32_t key, uint32_t place) {
        const uint32_t part = place / kEach >> 6;
        double unused;
        const uint64_t mass = kept(key, &unused);
        if (mass) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.mass[part]), static_cast<unsigned long long>(mass));
        if (key == border) atomicAdd(&sh.count[part], 1u);
      });
    }
  } else row.each([&](int c, const uint32_t (&w)[4]) {
    uint64_t mass = 0;
    uint32_t same = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const uint32_t key = L::key(bits_of<T>(w, e));
      double unused;
      mass += kept(key, &unused);
      same += key == border && border != L::kLowest;
    }
    mass = wave_sum64(mass);
    same = uint32_t(wave_sum64(same));
    const int part = c >> 6;
    if (lane == 0 && part < parts) {
      sh.mass[part] = mass;
      sh.count[part] = same;
    }
  });
  __syncthreads();
  {
    const int per = (parts + kThreads - 1) / kThreads;
    const int from = min(tid * per, parts), to = min(from + per, parts);
    uint64_t own = 0, all;
    for (int i = from; i < to; ++i) own += sh.count[i];
    uint64_t at = block_before(sh, own, &all);
    for (int i = from; i < to; ++i) {
      const uint64_t same = sh.count[i];
      const uint64_t take = at < ties ? min(ties - at, same) : 0;
      sh.mass[i] += take * border_units;
      sh.count[i] = uint32_t(at);               // those before the stretch
      at += same;
    }
  }
  __syncthreads();
  uint64_t before, target, total;
  const int part = find(sh, parts, [&](int i) { return sh.mass[i]; }, target_of, &before, &target, &total);
  if (wave != 0 || part < 0) return;
  target -= before;

  // the drawn token in its stretch
  const int c = part * 64 + lane;
  const uint4 v = row.load(c);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t key[kEach], same = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    key[e] = L::key(bits_of<T>(w, e));
    same += key[e] == border && border != L::kLowest;
  }
  uint32_t rank = uint32_t(wave_upto(same)) + sh.count[part] - same;    // equal tokens before this lane's
  uint64_t mass[kEach], own = 0;
  double exact[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    mass[e] = kept(key[e], &exact[e]);
    if (key[e] == border && border != L::kLowest) {
      exact[e] = border_weight;
      if (rank < ties) mass[e] = border_units;
      ++rank;
    }
    own += mass[e];
  }
  const uint64_t upto = wave_upto(own);
  uint64_t at = upto - own;
  if (at < target && target <= upto) {
    bool done = false;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      at += mass[e];
      if (!done && target <= at) {
        done = true;
        finish(c * kEach + e, float(exact[e] / double(total)));
      }
    }
  }
}

}  // namespace

hipError_t launch_sample(const SampleParams& p, hipStream_t stream) {
  SampleParams a = p;
  void* args[] = {&a};
  auto launch = [&](const void* fn32, const void* fn16, long wgs, int threads) {
    return hipLaunchKernel(p.f32 ? fn32 : fn16, dim3(unsigned(wgs)), dim3(unsigned(threads)), args, 0, stream);
  };
  if (p.maxima) {
    hipError_t e = launch(reinterpret_cast<const void*>(&sample_max_kernel<uint32_t>),
                          reinterpret_cast<const void*>(&sample_max_kernel<uint16_t>), long(p.rows) * p.blocks, kAheadThreads);
    if (e == hipSuccess && p.sums)
      e = launch(reinterpret_cast<const void*>(&sample_sum_kernel<uint32_t>),
                 reinterpret_cast<const void*>(&sample_sum_kernel<uint16_t>), long(p.rows) * p.blocks, kAheadThreads);
    if (e == hipSuccess && p.bins)
      e = launch(reinterpret_cast<const void*>(&sample_split_kernel<uint32_t>),
                 reinterpret_cast<const void*>(&sample_split_kernel<uint16_t>), long(p.rows) * p.blocks, kAheadThreads);
    if (e != hipSuccess) return e;
  }
  return launch(reinterpret_cast<const void*>(&sample_kernel<uint32_t>),
                reinterpret_cast<const void*>(&sample_kernel<uint16_t>), p.rows, kThreads);
}

}  // namespace w4a8
