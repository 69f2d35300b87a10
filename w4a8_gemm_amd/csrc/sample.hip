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

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "quant_common.h"
#include "verify_kernels.h"

namespace w4a8 {
namespace {

using namespace dev;

constexpr int kThreads = 1024;
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
  static constexpr uint32_t kLowest = 0x03FF;
  static __device__ __forceinline__ uint32_t key(uint32_t b) {
    b = b == 0x8000u ? 0u : b;
    return b & 0x8000u ? ~b & 0xFFFFu : b | 0x8000u;
  }
  static __device__ __forceinline__ double value(uint32_t key) {
    return double(h2f(uint16_t(key & 0x8000u ? key ^ 0x8000u : ~key)));
  }
  static __device__ __forceinline__ bool bad(uint32_t b) { return (b & 0x7FFFu) >= 0x7C00u && b != 0xFC00u; }
};
template <>
struct Logit<uint32_t> {
  static constexpr int kBits = 32, kEach = 4;
  static constexpr uint32_t kLowest = 0x007FFFFF;
  static __device__ __forceinline__ uint32_t key(uint32_t b) {
    b = b == 0x80000000u ? 0u : b;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
  }
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
  const T* from;              // the aligned bytes that hold the first logit
  int head, end;              // its place there, and the place behind the last
  __device__ __forceinline__ int chunks() const { return (end + Logit<T>::kEach - 1) / Logit<T>::kEach; }
  // the keys of chunk c, kLowest where there is no logit; *bad if one is NaN or
  // infinite
  __device__ __forceinline__ void load(int c, uint32_t (&key)[Logit<T>::kEach], bool* bad) const {
    constexpr int kEach = Logit<T>::kEach;
    const int at = c * kEach;
    T raw[kEach];
    if (at >= head && at + kEach <= end) {
      __builtin_memcpy(raw, __builtin_assume_aligned(from + at, 16), 16);
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        key[e] = Logit<T>::key(raw[e]);
        *bad |= Logit<T>::bad(raw[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        key[e] = Logit<T>::kLowest;
        if (at + e >= head && at + e < end) {
          const uint32_t b = from[at + e];
          key[e] = Logit<T>::key(b);
          *bad |= Logit<T>::bad(b);
        }
      }
    }
  }
};

struct Shared {
  uint64_t mass[kParts];      // of bins, then of stretches
  uint32_t count[kParts];
  uint64_t sums[kWaves];
  uint64_t found_before;
  int found;
};

__device__ __forceinline__ uint64_t shfl_up64(uint64_t x, int d) {
  const uint32_t lo = __shfl_up(uint32_t(x), d), hi = __shfl_up(uint32_t(x >> 32), d);
  return lo | uint64_t(hi) << 32;
}

// Sums of the threads before this one; *total that of all.  All threads call it.
__device__ __forceinline__ uint64_t block_before(Shared& sh, uint64_t x, uint64_t* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint64_t upto = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t y = shfl_up64(upto, d);
    if (lane >= d) upto += y;
  }
  __syncthreads();                        // the last call's sums have been read
  if (lane == 63) sh.sums[wave] = upto;
  __syncthreads();
  uint64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += sh.sums[w];
    all += sh.sums[w];
  }
  *total = all;
  return before + upto - x;
}

// The first i of n for which the values up to it reach the target, and the sum
// before it; -1 if their total does not.  The target (1 or more) is given for
// the total.  All threads call it and get the same.
template <typename Value, typename Target>
__device__ __forceinline__ int find(Shared& sh, int n, Value value, Target target_of, uint64_t* before,
                                    uint64_t* target, uint64_t* total) {
  const int per = (n + kThreads - 1) / kThreads;
  const int from = min(int(threadIdx.x) * per, n), to = min(from + per, n);
  uint64_t mine = 0;
  for (int i = from; i < to; ++i) mine += value(i);
  if (threadIdx.x == 0) sh.found = -1;
  uint64_t at = block_before(sh, mine, total);
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

template <typename T>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleParams p) {
  using L = Logit<T>;
  constexpr int kEach = L::kEach;
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const long r = blockIdx.x;
  Row<T> row;
  {
    const T* at = static_cast<const T*>(p.logits) + r * p.ld;
    row.head = int((reinterpret_cast<uintptr_t>(at) & 15u) / sizeof(T));
    row.from = at - row.head;
    row.end = row.head + p.vocab;
  }
  const int chunks = row.chunks();
  const float temperature = p.s.temperature_dev ? p.s.temperature_dev[r] : p.s.temperature;
  const int top_k = p.s.top_k_dev ? p.s.top_k_dev[r] : p.s.top_k;
  const float top_p = p.s.top_p_dev ? p.s.top_p_dev[r] : p.s.top_p;
  const float min_p = p.s.min_p_dev ? p.s.min_p_dev[r] : p.s.min_p;
  const float u_raw = p.u[r];

  auto finish = [&](int token, float prob) {
    p.tokens[r] = token;
    if (p.probs) p.probs[r] = prob;
  };

  // the largest logit
  bool bad = !(temperature >= 0.0f) || temperature == __builtin_inff() || top_p != top_p || min_p != min_p;
  uint32_t top = L::kLowest;
  for (int c = tid; c < chunks; c += kThreads) {
    uint32_t key[kEach];
    row.load(c, key, &bad);
#pragma unroll
    for (int e = 0; e < kEach; ++e) top = max(top, key[e]);
  }
  top = wave_max_u32(top);
  const bool wave_bad = __ballot(bad) != 0;
  if (lane == 0) sh.sums[wave] = top | uint64_t(wave_bad) << 32;
  __syncthreads();
  bad = false;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    top = max(top, uint32_t(sh.sums[w]));
    bad |= sh.sums[w] >> 32 != 0;
  }
  if (bad || top == L::kLowest) {
    if (tid == 0) finish(-1, bad ? __builtin_nanf("") : 0.0f);
    return;
  }

  // the first token with it
  if (temperature == 0.0f || top_k == 1) {
    uint32_t none = 0;                      // largest of ~place
    for (int c = tid; c < chunks; c += kThreads) {
      uint32_t key[kEach];
      row.load(c, key, &bad);
#pragma unroll
      for (int e = kEach - 1; e >= 0; --e)
        if (key[e] == top) none = max(none, ~uint32_t(c * kEach + e));
    }
    none = wave_max_u32(none);
    __syncthreads();
    if (lane == 0) sh.sums[wave] = none;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) none = max(none, uint32_t(sh.sums[w]));
    if (tid == 0) finish(int(~none) - row.head, 1.0f);
    return;
  }

  // weights, as multiples of 2^-44 before and after rounding
  const double largest = L::value(top), turn = 1.4426950408889634 / double(temperature);
  auto weight = [&](uint32_t key) -> double {
    const double t = (L::value(key) - largest) * turn;
    if (!(t > -64.0)) return 0.0;
    const double whole = __builtin_rint(t);
    return __builtin_ldexp(exp2_near0(t - whole), int(whole) + kUnitBits);
  };
  auto units = [](double w) -> uint64_t {
    return __builtin_bit_cast(uint64_t, w + 0x1p52) & ((1ull << 52) - 1);
  };
  const double least = double(min_p > 0.0f ? fminf(min_p, 1.0f) : 0.0f) * (1ull << kUnitBits);

  // The tokens kept: keys above `border`, and the first `ties` that have it.
  uint32_t border = L::kLowest;
  uint64_t ties = 0;
  // Finds the key at which the counts (MASS: the weights) of the tokens kept so
  // far, added from the largest key down, reach the target; what is left of the
  // target there.
  auto select = [&](auto mass_tag, auto target_of, uint32_t* key_out, uint64_t* left) {
    constexpr bool kMass = decltype(mass_tag)::value;
    uint32_t prefix = 0;
    uint64_t target = 0;
    const uint64_t border_mass = kMass && ties ? ties * units(weight(border)) : 0;
#pragma unroll
    for (int shift = L::kBits, width; shift > 0; shift -= width) {
      width = min(kBinBits, shift);
      const bool first = shift == L::kBits;
      const int low = shift - width;
      __syncthreads();
      for (int i = tid; i < kBins; i += kThreads) {
        if (kMass) sh.mass[i] = 0;
        else sh.count[i] = 0;
      }
      __syncthreads();
      auto bin_of = [&](uint32_t key) { return key >> low & ((1u << width) - 1); };
      auto inside = [&](uint32_t key) { return first || key >> (shift & 31) == prefix; };
      for (int c = tid; c < chunks; c += kThreads) {
        uint32_t key[kEach];
        bool unused = false;
        row.load(c, key, &unused);
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          if (key[e] <= border || !inside(key[e])) continue;
          if constexpr (kMass)
            atomicAdd(reinterpret_cast<unsigned long long*>(&sh.mass[bin_of(key[e])]), units(weight(key[e])));
          else
            atomicAdd(&sh.count[bin_of(key[e])], 1u);
        }
      }
      if (kMass && tid == 0 && border_mass && inside(border))
        atomicAdd(reinterpret_cast<unsigned long long*>(&sh.mass[bin_of(border)]), border_mass);
      __syncthreads();
      const int n = 1 << width;
      uint64_t before, total;
      const int at = find(sh, n, [&](int i) { return kMass ? sh.mass[n - 1 - i] : uint64_t(sh.count[n - 1 - i]); },
                          [&](uint64_t all) { return first ? target_of(all) : target; }, &before, &target, &total);
      if (at < 0) return false;
      target -= before;
      prefix = prefix << width | uint32_t(n - 1 - at);
    }
    *key_out = prefix;
    *left = target;
    return true;
  };
  if (top_k > 0 && top_k < p.vocab) {
    uint32_t key;
    uint64_t left;
    if (select(std::false_type(), [&](uint64_t) { return uint64_t(top_k); }, &key, &left)) {
      border = key;
      ties = left;
    }
  }
  if (top_p < 1.0f) {
    uint32_t key;
    uint64_t left;
    auto share = [&](uint64_t all) {
      const double want = __builtin_ceil(double(fmaxf(top_p, 0.0f)) * double(all));
      return max(uint64_t(want), uint64_t(1));
    };
    if (select(std::true_type(), share, &key, &left)) {
      const uint64_t each = units(weight(key));
      border = key;
      ties = (left + each - 1) / each;
    }
  }
  const double border_weight = weight(border);
  const uint64_t border_units = units(border_weight);
  if (border == L::kLowest || border_weight < least) ties = 0;

  // kept weight of every stretch of 64 chunks, without and then with the tokens
  // at the border
  auto kept = [&](uint32_t key, double* w) -> uint64_t {
    if (key <= border) return 0;
    *w = weight(key);
    return *w >= least ? units(*w) : 0;
  };
  const int parts = (chunks + 63) / 64;
  __syncthreads();
  for (int part = wave; part < parts; part += kWaves) {
    uint32_t key[kEach];
    bool unused = false;
    const int c = part * 64 + lane;
#pragma unroll
    for (int e = 0; e < kEach; ++e) key[e] = L::kLowest;
    if (c < chunks) row.load(c, key, &unused);
    uint64_t mass = 0;
    uint32_t same = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      double w;
      mass += kept(key[e], &w);
      same += key[e] == border && border != L::kLowest;
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
      mass += uint64_t(__shfl_xor(uint32_t(mass), d)) | uint64_t(__shfl_xor(uint32_t(mass >> 32), d)) << 32;
      same += __shfl_xor(same, d);
    }
    if (lane == 0) {
      sh.mass[part] = mass;
      sh.count[part] = same;
    }
  }
  __syncthreads();
  {
    const int per = (parts + kThreads - 1) / kThreads;
    const int from = min(tid * per, parts), to = min(from + per, parts);
    uint64_t mine = 0, all;
    for (int i = from; i < to; ++i) mine += sh.count[i];
    uint64_t at = block_before(sh, mine, &all);
    for (int i = from; i < to; ++i) {
      const uint64_t same = sh.count[i];
      const uint64_t take = at < ties ? min(ties - at, same) : 0;
      sh.mass[i] += take * border_units;
      sh.count[i] = uint32_t(at);               // those before the stretch
      at += same;
    }
  }
  __syncthreads();
  const float u = u_raw >= 0.0f ? fminf(u_raw, 0x1.fffffep-1f) : 0.0f;
  uint64_t before, target, total;
  const int part = find(sh, parts, [&](int i) { return sh.mass[i]; },
                        [&](uint64_t all) { return uint64_t(double(u) * double(all)) + 1; }, &before, &target, &total);
  if (wave != 0 || part < 0) return;
  target -= before;

  // the drawn token in its stretch
  uint32_t key[kEach];
  bool unused = false;
  const int c = part * 64 + lane;
#pragma unroll
  for (int e = 0; e < kEach; ++e) key[e] = L::kLowest;
  if (c < chunks) row.load(c, key, &unused);
  uint32_t same = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) same += key[e] == border && border != L::kLowest;
  uint32_t rank = same;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t y = __shfl_up(rank, d);
    if (lane >= d) rank += y;
  }
  rank += sh.count[part] - same;                // equal tokens before this lane's
  uint64_t w[kEach], mine = 0;
  double exact[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    w[e] = kept(key[e], &exact[e]);
    if (key[e] == border && border != L::kLowest) {
      exact[e] = border_weight;
      if (rank < ties) w[e] = border_units;
      ++rank;
    }
    mine += w[e];
  }
  uint64_t upto = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t y = shfl_up64(upto, d);
    if (lane >= d) upto += y;
  }
  uint64_t at = upto - mine;
  if (at < target && target <= upto) {
    bool done = false;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      at += w[e];
      if (!done && target <= at) {
        done = true;
        finish(c * kEach + e - row.head, float(exact[e] / double(total)));
      }
    }
  }
}

}  // namespace

hipError_t launch_sample(const SampleParams& p, hipStream_t stream) {
  SampleParams a = p;
  void* args[] = {&a};
  const void* fn = p.f32 ? reinterpret_cast<const void*>(&sample_kernel<uint32_t>)
                         : reinterpret_cast<const void*>(&sample_kernel<uint16_t>);
  return hipLaunchKernel(fn, dim3(unsigned(p.rows)), dim3(kThreads), args, 0, stream);
}

}  // namespace w4a8
