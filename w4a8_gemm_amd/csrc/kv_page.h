// Device helpers shared by the append and the attention over the paged int8
// cache: which sequence a virtual index belongs to, and where a page lies.
//
// Everything read from device memory (lengths, offsets, page numbers) is
// clamped to the bounds the host checked, so that no content of those tables
// can take a kernel outside its buffers.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "decoder_kernels.h"

namespace w4a8 {
namespace kv {

// A sequence's new tokens [lo, hi) among all new tokens, and its length with
// them.  The position of new token t is len - (hi - lo) + (t - lo).
struct Seq {
  int lo, hi, len;
};

static __device__ __forceinline__ Seq seq_of(const KvArgs& a, int b) {
  Seq s;
  if (a.cu_q) {
    s.lo = min(max(a.cu_q[b], 0), a.total_q);
    s.hi = min(max(a.cu_q[b + 1], s.lo), a.total_q);
  } else {
    s.lo = b;
    s.hi = b + 1;
  }
  // max_pages << page_shift fits an int (host check)
  s.len = min(max(a.lens[b], 0), a.max_pages << a.page_shift);
  return s;
}

// The largest b with first(b) <= w, for an ascending first: the sequence that
// owns virtual index w; *index is w's place in it.
// first(0) is 0 for a proper cu_q; an improper one gives some sequence in range.
template <typename First>
static __device__ __forceinline__ int owner(int w, int batch, First first, int* index) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first(mid) <= w)
      lo = mid;
    else
      hi = mid - 1;
  }
  *index = w - first(lo);
  return lo;
}

// page number `i` of sequence b, or -1 where the table holds none
static __device__ __forceinline__ int page_at(const KvArgs& a, int b, int i) {
  if (i < 0 || i >= a.max_pages) return -1;
  const int p = a.table[long(b) * a.table_ld + i];
  return p >= 0 && p < a.num_pages ? p : -1;
}

// The keys of split `split` among [lo, hi): chunk keys from split * chunk on
// (the last split takes all that follow).
struct Range {
  int lo, hi;
};
static __device__ __forceinline__ Range split_range(int split, int splits, int chunk, int lo,
                                                    int hi) {
  const long from = long(split) * chunk;
  Range r;
  r.lo = int(max(long(lo), min(from, long(hi))));
  r.hi = split == splits - 1 ? hi : int(min(long(hi), from + chunk));
  return r;
}

// 4-byte load from an address all lanes share, through the scalar cache
static __device__ __forceinline__ int scalar_load(const int32_t* p) {
  return *(const __attribute__((address_space(4))) int32_t*)(uintptr_t(p));
}

}  // namespace kv
}  // namespace w4a8
