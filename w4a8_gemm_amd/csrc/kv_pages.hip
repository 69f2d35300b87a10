// Pages of a paged cache that sequences share (gfx950): reference counts and
// tables for sequences that continue others, fresh pages for next tokens, the
// pages in use moved together, and copies of pages.
//
// The tables are int32 and every result is one of whole numbers that does not
// depend on scheduling: atomics only count, or keep a largest row, and free pages
// are handed out in ascending order to requests in the order of sequences and
// positions.  Latency bounds the table operators; copies are bound by memory.
// Measured: 64 beams in groups of 4 over 500 tokens in pages of 16, forked 5.5 us (two
// launches), given pages 10.7 (three; the scan over rows, one workgroup, 4.9), 1 MB of
// shared pages copied 3.7; pages of 16 for a prompt of 8192 tokens 60 (a page a turn of
// the row's wave, 0.1 each), for 16 of 2000 26; half of a pool of 1500 pages of 64 KB
// moved together 12.5 (three) and 24.6 MB of it copied 9.6 us, 5.1 TB/s read and written.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kv_page.h"
#include "quant_common.h"
#include "verify_kernels.h"

namespace w4a8 {
namespace {

constexpr int kThreads = 256;
constexpr int kScanThreads = 1024;

// A table's entry, -1 for any that names no page of the pool.
__device__ __forceinline__ int entry(const TableArgs& t, int row, int column) {
  const int p = t.table[long(row) * t.table_ld + column];
  return p >= 0 && p < t.num_pages ? p : -1;
}

__device__ __forceinline__ int length_of(const int32_t* lens, int b, const TableArgs& t, int shift) {
  return min(max(lens[b], 0), t.max_pages << shift);
}

// Sums of the values of the threads before this one; *total that of all.  Every
// thread of the workgroup calls it.
template <int THREADS, typename Sum = int>
__device__ __forceinline__ Sum block_before(Sum x, Sum* total) {
  constexpr int kW = THREADS / 64;
  __shared__ Sum sums[kW];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  Sum upto = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const Sum y = __shfl_up(upto, d);
    if (lane >= d) upto += y;
  }
  __syncthreads();                       // the last call's sums have been read
  if (lane == 63) sums[wave] = upto;
  __syncthreads();
  Sum before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kW; ++w) {
    if (w < wave) before += sums[w];
    all += sums[w];
  }
  *total = all;
  return before + upto - x;
}

// ------------------------------------------------------------------- fork
// Row i of the new table continues row parent[i]: all pages of its own row, the
// pages with tokens of another.
__device__ __forceinline__ int forked(const ForkParams& p, int row, int column) {
  const int from = p.parent[row];
  if (from < 0 || from >= p.t.batch) return -1;
  if (from != row) {
    const int len = length_of(p.lens, from, p.t, p.page_shift);
    if (column >= (len + (1 << p.page_shift) - 1) >> p.page_shift) return -1;
  }
  return entry(p.t, from, column);
}

__global__ __launch_bounds__(kThreads) void fork_kernel(ForkParams p) {
  const long i = long(blockIdx.x) * kThreads + threadIdx.x;
  if (i < long(p.new_batch) * p.t.max_pages) {
    const int row = int(i / p.t.max_pages), column = int(i - long(row) * p.t.max_pages);
    p.t.new_table[row * p.t.new_ld + column] = forked(p, row, column);
  }
  if (i < p.t.num_pages) p.t.new_refs[i] = p.t.refs[i];
  if (i < p.new_batch) {
    const int from = p.parent[i];
    p.new_lens[i] = from >= 0 && from < p.t.batch ? p.lens[from] : 0;
  }
}

// Entries that go and entries that come; rows that stay as they are do neither.
__global__ __launch_bounds__(kThreads) void fork_refs_kernel(ForkParams p) {
  const long i = long(blockIdx.x) * kThreads + threadIdx.x;
  const int rows = max(p.t.batch, p.new_batch);
  if (i >= long(rows) * p.t.max_pages) return;
  const int row = int(i / p.t.max_pages), column = int(i - long(row) * p.t.max_pages);
  const bool stays = row < p.new_batch && row < p.t.batch && p.parent[row] == row;
  if (stays) return;
  if (row < p.t.batch) {
    const int page = entry(p.t, row, column);
    if (page >= 0) atomicSub(&p.t.new_refs[page], 1);
  }
  if (row < p.new_batch) {
    const int page = forked(p, row, column);
    if (page >= 0) atomicAdd(&p.t.new_refs[page], 1);
  }
}

// ------------------------------------------------------------------ alloc
struct Span {
  int first, end;             // entries that get tokens
  bool half;                  // the first has earlier tokens
  int over;                   // entries beyond the table
};

__device__ __forceinline__ Span span_of(const AllocParams& p, int b) {
  const int page = 1 << p.page_shift;
  const int len = length_of(p.lens, b, p.t, p.page_shift);
  const int tokens = max(p.tokens_dev ? p.tokens_dev[b] : p.tokens, 0);
  const long end = (long(len) + tokens + page - 1) >> p.page_shift;
  Span s;
  s.first = len >> p.page_shift;
  s.end = int(min(end, long(p.t.max_pages)));
  s.half = (len & (page - 1)) != 0 && tokens > 0;
  s.over = int(end - s.end);
  if (tokens == 0) s.end = s.first;
  return s;
}

// One workgroup a row: its entries copied, those that need a page counted.  Then
// one a block of pages: counts copied, free ones counted.
__global__ __launch_bounds__(kThreads) void alloc_count_kernel(AllocParams p) {
  if (int(blockIdx.x) >= p.t.batch) {
    const int block = int(blockIdx.x) - p.t.batch;
    int free = 0, total;
#pragma unroll
    for (int k = 0; k < kPageBlock; k += kThreads) {
      const int page = block * kPageBlock + k + int(threadIdx.x);
      if (page < p.t.num_pages) {
        const int refs = p.t.refs[page];
        p.t.new_refs[page] = refs;
        p.writers[page] = 0;
        p.final_row[page] = -1;
        free += refs <= 0;
      }
    }
    block_before<kThreads>(free, &total);
    if (threadIdx.x == 0) p.block_free[block] = total;
    return;
  }
  const int b = int(blockIdx.x);
  const Span s = span_of(p, b);
  int need = 0, total;
  for (int column = threadIdx.x; column < p.t.max_pages; column += kThreads) {
    const int page = entry(p.t, b, column);
    p.t.new_table[b * p.t.new_ld + column] = page;
    need += page < 0 && column >= s.first && column < s.end;
  }
  block_before<kThreads>(need, &total);
  if (threadIdx.x == 0) {
    const int tokens = max(p.tokens_dev ? p.tokens_dev[b] : p.tokens, 0);
    p.new_lens[b] = int(min(long(length_of(p.lens, b, p.t, p.page_shift)) + tokens, 2147483647l));
    p.row_need[b] = total;
    p.row_held[b] = s.half && s.first < p.t.max_pages ? entry(p.t, b, s.first) : -1;
    p.row_over[b] = s.over;
  }
}

// One workgroup: which sequences copy the page that they go on writing, and where
// each one's requests begin.  A shared page is copied by all that write it,
// except by the last of them if nobody else holds it.
__global__ __launch_bounds__(kScanThreads) void alloc_scan_kernel(AllocParams p, int blocks) {
  const int tid = threadIdx.x;
  int free = 0, all;
  for (int base = 0; base < blocks; base += kScanThreads) {
    const int i = base + tid;
    const int x = i < blocks ? p.block_free[i] : 0;
    const int before = block_before<kScanThreads>(x, &all);
    if (i < blocks) p.block_free[i] = free + before;
    free += all;
  }
  for (int b = tid; b < p.t.batch; b += kScanThreads) {
    const int page = p.row_held[b];
    if (page >= 0) {
      atomicAdd(&p.writers[page], 1);
      atomicMax(&p.final_row[page], b);
    }
  }
  __syncthreads();
  int requests = 0, pairs = 0;
  long beyond = 0;                        // a row of 2^31 - 1 tokens counts 2^27
  for (int base = 0; base < p.t.batch; base += kScanThreads) {
    const int b = base + tid;
    int copies = 0, need = 0;
    if (b < p.t.batch) {
      const int page = p.row_held[b];
      need = p.row_need[b];
      beyond += p.row_over[b];
      if (page >= 0) {
        const int refs = p.t.refs[page];
        const int writers = __hip_atomic_load(&p.writers[page], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const int final_row = __hip_atomic_load(&p.final_row[page], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        copies = refs > 1 && !(writers >= refs && final_row == b);
      }
    }
    const int before = requests + block_before<kScanThreads>(need + copies, &all);
    requests += all;
    const bool gets = copies && before < free;           // a row's copy is its first request
    const int place = pairs + block_before<kScanThreads>(gets ? 1 : 0, &all);
    pairs += all;
    if (b < p.t.batch) {
      p.row_base[b] = before;
      p.row_pair[b] = gets ? place : -1;
      if (!copies) p.row_held[b] = -1;
    }
  }
  for (int i = pairs + tid; i < p.t.batch; i += kScanThreads) {
    p.src[i] = -1;
    p.dst[i] = -1;
  }
  long missing = 0;
  if (__syncthreads_or(beyond != 0)) block_before<kScanThreads>(beyond, &missing);
  if (tid == 0) {
    p.counts[0] = pairs;
    p.counts[1] = int(min(missing + max(requests - free, 0), 2147483647l));
  }
}

// One wave a row: its requests take the free pages from place row_base on.  The
// counts as they were say which pages are free; the new ones are only written.
__global__ __launch_bounds__(kThreads) void alloc_hand_kernel(AllocParams p, int blocks) {
  const int lane = threadIdx.x & 63;
  const int b = int(blockIdx.x) * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (b >= p.t.batch) return;
  const Span s = span_of(p, b);
  const int held = p.row_held[b];
  int need = p.row_need[b] + (held >= 0);
  if (need == 0) return;
  int32_t* const row = p.t.new_table + b * p.t.new_ld;
  // the block of pages that holds the first of them
  int lo = 0, hi = blocks - 1;
  const int want = p.row_base[b];
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.block_free[mid] <= want) lo = mid;
    else hi = mid - 1;
  }
  int skip = want - p.block_free[lo];                // free pages before it there
  int at = lo * kPageBlock;                          // pages looked at from here on
  uint64_t ready = 0;                                // free ones among 64 not handed out yet
  int ready_at = 0;
  auto next = [&]() {
    while (!ready) {
      if (at >= p.t.num_pages) return -1;
      const int page = at + lane;
      uint64_t free = __ballot(page < p.t.num_pages && p.t.refs[page] <= 0);
      ready_at = at;
      at += 64;
      const int here = __builtin_popcountll(free);
      if (skip >= here) {
        skip -= here;
        continue;
      }
      for (; skip > 0; --skip) free &= free - 1;
      ready = free;
    }
    const int page = ready_at + __builtin_ctzll(ready);
    ready &= ready - 1;
    return page;
  };
  if (held >= 0) {
    const int page = next();
    const int pair = p.row_pair[b];
    if (lane == 0) {
      row[s.first] = page;
      atomicSub(&p.t.new_refs[held], 1);
      if (page >= 0) p.t.new_refs[page] = 1;
      if (pair >= 0) {
        p.src[pair] = held;
        p.dst[pair] = page;
      }
    }
    --need;
  }
  for (int base = s.first; base < s.end && need > 0; base += 64) {
    const int column = base + lane;
    uint64_t empty = __ballot(column < s.end && entry(p.t, b, column) < 0);
    for (; empty; empty &= empty - 1) {
      const int page = next();
      --need;
      if (page < 0) return;                          // the rest stays without one
      if (lane == 0) {
        row[base + __builtin_ctzll(empty)] = page;
        p.t.new_refs[page] = 1;
      }
    }
  }
}

// ---------------------------------------------------------------- compact
// With `live` pages in use, the n-th of them at `live` or beyond goes to the n-th
// free page before.
__global__ __launch_bounds__(kThreads) void compact_count_kernel(CompactParams p) {
  int live = 0, total;
#pragma unroll
  for (int k = 0; k < kPageBlock; k += kThreads) {
    const int page = int(blockIdx.x) * kPageBlock + k + int(threadIdx.x);
    live += page < p.t.num_pages && p.t.refs[page] > 0;
  }
  block_before<kThreads>(live, &total);
  if (threadIdx.x == 0) p.block_live[blockIdx.x] = total;
}

// pages in use: of all blocks, and of those before block `upto`
__device__ __forceinline__ void live_of(const CompactParams& p, int blocks, int upto, int* live, int* before) {
  int all = 0, part = 0;
  for (int i = threadIdx.x; i < blocks; i += kThreads) {
    const int x = p.block_live[i];
    all += x;
    part += i < upto ? x : 0;
  }
  block_before<kThreads>(all, live);
  block_before<kThreads>(part, before);
}

__global__ __launch_bounds__(kThreads) void compact_rank_kernel(CompactParams p, int blocks) {
  const int block = int(blockIdx.x);
  int live, before, unused;
  live_of(p, blocks, block, &live, &before);
  // those before page `live`: of the blocks before its block, and in it
  int ahead;
  live_of(p, blocks, live / kPageBlock, &unused, &ahead);
  int part = 0, inside;
#pragma unroll
  for (int k = 0; k < kPageBlock; k += kThreads) {
    const int page = live / kPageBlock * kPageBlock + k + int(threadIdx.x);
    part += page < live && page < p.t.num_pages && p.t.refs[page] > 0;
  }
  block_before<kThreads>(part, &inside);
  ahead += inside;
  const int moves = live - ahead;
  if (block == 0 && threadIdx.x == 0) {
    p.counts[0] = moves;
    p.counts[1] = 0;
  }
#pragma unroll
  for (int k = 0; k < kPageBlock; k += kThreads) {
    const int page = block * kPageBlock + k + int(threadIdx.x);
    const bool used = page < p.t.num_pages && p.t.refs[page] > 0;
    const int upto = before + block_before<kThreads>(used ? 1 : 0, &unused);
    before += unused;
    if (page >= p.t.num_pages) continue;
    int rank = -1;
    if (used && page >= live) {
      rank = upto - ahead;
      p.src[rank] = page;
    } else if (!used && page < live) {
      rank = page - upto;
      p.dst[rank] = page;
    }
    p.rank[page] = rank;
  }
}

__global__ __launch_bounds__(kThreads) void compact_apply_kernel(CompactParams p) {
  const long i = long(blockIdx.x) * kThreads + threadIdx.x;
  // a page that moves is one with a rank that is in use
  auto place_of = [&](int page) {
    const int rank = p.rank[page];
    return rank >= 0 && p.t.refs[page] > 0 ? p.dst[rank] : page;
  };
  if (i < long(p.t.batch) * p.t.max_pages) {
    const int row = int(i / p.t.max_pages), column = int(i - long(row) * p.t.max_pages);
    const int page = entry(p.t, row, column);
    p.t.new_table[row * p.t.new_ld + column] = page >= 0 ? place_of(page) : -1;
  }
  if (i < p.t.num_pages) {
    const int page = int(i), rank = p.rank[page], refs = p.t.refs[page];
    p.place[page] = place_of(page);
    p.t.new_refs[page] = rank < 0 ? max(refs, 0) : refs > 0 ? 0 : p.t.refs[p.src[rank]];
  }
  const int moves = p.counts[0];
  if (i >= moves && i < p.t.num_pages / 2) {
    p.src[i] = -1;
    p.dst[i] = -1;
  }
}

// ------------------------------------------------------------------- copy
// 4096 bytes a step of a workgroup, pairs after pairs.
constexpr int kCopyBytes = kThreads * 16;

__global__ __launch_bounds__(kThreads) void copy_kernel(CopyParams p, int parts) {
  const long pairs = p.count ? min(max(p.count[0], 0), p.pairs) : p.pairs;
  for (long i = blockIdx.x; i < pairs * parts; i += gridDim.x) {
    const int pair = int(i / parts), part = int(i - long(pair) * parts);
    const int from = kv::scalar_load(p.src + pair), to = kv::scalar_load(p.dst + pair);
    if (from < 0 || from >= p.num_pages || to < 0 || to >= p.num_pages) continue;
    const int at = part * kCopyBytes + int(threadIdx.x) * 16;
    if (at < p.page_bytes)
      *reinterpret_cast<uint4*>(p.data + to * p.page_stride + at) =
          *reinterpret_cast<const uint4*>(p.data + from * p.page_stride + at);
    if (part == 0)
      for (int s = threadIdx.x; s < p.scales; s += kThreads)
        p.scale[to * p.scale_stride + s] = p.scale[from * p.scale_stride + s];
  }
}

unsigned blocks_of(long items, int each) { return unsigned((items + each - 1) / each); }

}  // namespace

hipError_t launch_kv_fork(const ForkParams& p, hipStream_t stream) {
  ForkParams a = p;
  void* args[] = {&a};
  const long items = std::max({long(p.new_batch) * p.t.max_pages, long(p.t.num_pages), 1l});
  hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&fork_kernel), dim3(blocks_of(items, kThreads)),
                                 dim3(kThreads), args, 0, stream);
  const long entries = long(std::max(p.t.batch, p.new_batch)) * p.t.max_pages;
  if (e != hipSuccess || entries == 0) return e;
  return hipLaunchKernel(reinterpret_cast<const void*>(&fork_refs_kernel), dim3(blocks_of(entries, kThreads)),
                         dim3(kThreads), args, 0, stream);
}

hipError_t launch_kv_alloc(const AllocParams& p, hipStream_t stream) {
  AllocParams a = p;
  int blocks = page_blocks(p.t.num_pages);
  void* args[] = {&a, &blocks};
  hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&alloc_count_kernel),
                                 dim3(unsigned(p.t.batch + blocks)), dim3(kThreads), args, 0, stream);
  if (e != hipSuccess) return e;
  e = hipLaunchKernel(reinterpret_cast<const void*>(&alloc_scan_kernel), dim3(1), dim3(kScanThreads), args, 0, stream);
  if (e != hipSuccess || p.t.batch == 0) return e;
  return hipLaunchKernel(reinterpret_cast<const void*>(&alloc_hand_kernel), dim3(blocks_of(p.t.batch, kThreads / 64)),
                         dim3(kThreads), args, 0, stream);
}

hipError_t launch_kv_compact(const CompactParams& p, hipStream_t stream) {
  CompactParams a = p;
  int blocks = page_blocks(p.t.num_pages);
  void* args[] = {&a, &blocks};
  hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&compact_count_kernel), dim3(unsigned(blocks)),
                                 dim3(kThreads), args, 0, stream);
  if (e != hipSuccess) return e;
  e = hipLaunchKernel(reinterpret_cast<const void*>(&compact_rank_kernel), dim3(unsigned(blocks)), dim3(kThreads),
                      args, 0, stream);
  if (e != hipSuccess) return e;
  const long items = std::max(long(p.t.batch) * p.t.max_pages, long(p.t.num_pages));
  return hipLaunchKernel(reinterpret_cast<const void*>(&compact_apply_kernel), dim3(blocks_of(items, kThreads)),
                         dim3(kThreads), args, 0, stream);
}

hipError_t launch_kv_copy(const CopyParams& p, hipStream_t stream) {
  CopyParams a = p;
  int parts = (p.page_bytes + kCopyBytes - 1) / kCopyBytes;
  void* args[] = {&a, &parts};
  const long wgs = std::min(long(p.pairs) * parts, 8192l);
  return hipLaunchKernel(reinterpret_cast<const void*>(&copy_kernel), dim3(unsigned(wgs)), dim3(kThreads), args, 0,
                         stream);
}

}  // namespace w4a8
