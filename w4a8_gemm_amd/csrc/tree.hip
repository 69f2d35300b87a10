// Trees of drafted tokens (gfx950): which tokens each may see, which of them the
// sampled tokens confirm, and the confirmed ones' keys and values moved together
// in the paged int8 cache.
//
// A sequence's drafted tokens are its last ones, parents before children; a
// parent outside [0, child) means none.  Node 0 is the root: the sequence's last
// certain token, whose sampled successor selects among its children.
//
// All three are latency: a launch and loads that wait for each other.  Measured,
// graph replays of tree_accept and kv_keep: one tree of 26 nodes, heads 32 / 8 of
// 128, 6.7 us (2.9 and 4.3 in the kernels); 96 of up to 64 nodes 10.7 (5.7 and 7.1),
// where the 1.9 MB that are read and written would take 0.4.  tree_mask: one tree of 26
// 2.7 us, 16 of 64 3.7, 64 chains of 64 12, 6 chains of 200 36 (a load a level).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kv_page.h"
#include "quant_common.h"
#include "verify_kernels.h"

namespace w4a8 {
namespace {

using namespace dev;

constexpr int kThreads = 256;

struct Nodes {
  int b, lo, n;
};

__device__ __forceinline__ Nodes nodes_of(const TreeBatch& t, int b) {
  Nodes s;
  s.b = b;
  if (t.cu_q) {
    s.lo = min(max(t.cu_q[b], 0), t.total_q);
    s.n = min(max(t.cu_q[b + 1], s.lo), t.total_q) - s.lo;
  } else {
    s.lo = b;
    s.n = 1;
  }
  return s;
}

// One thread a drafted token: it walks to its root, setting a bit for itself and
// each token that it passes.
__global__ __launch_bounds__(kThreads) void tree_mask_kernel(TreeMaskParams p) {
  const int token = int(blockIdx.x) * kThreads + threadIdx.x;
  if (token >= p.tree.total_q) return;
  int b = token, unused = 0;
  if (p.tree.cu_q)
    b = kv::owner(token, p.tree.batch, [&](int i) { return p.tree.cu_q[i]; }, &unused);
  const Nodes s = nodes_of(p.tree, b);
  if (token < s.lo || token >= s.lo + s.n) return;    // behind the last sequence
  uint32_t* row = p.mask + long(token) * p.mask_ld;
  for (int w = 0; w < p.words; ++w) row[w] = 0;
  int node = token - s.lo, depth = 0, w = node >> 5;
  uint32_t bits = 0;
  for (;;) {
    if (node >> 5 != w) {
      if (w < p.words) row[w] = bits;
      w = node >> 5;
      bits = 0;
    }
    bits |= 1u << (node & 31);
    const int up = p.tree.parents[s.lo + node];
    if (up < 0 || up >= node) break;
    node = up;
    ++depth;
  }
  if (w < p.words) row[w] = bits;
  if (p.positions) p.positions[token] = p.tree.lens[b] - s.n + depth;
}

// One wave a sequence.  Each step looks for the first child of the current node
// that holds the token sampled there, 64 nodes at a time.
__global__ __launch_bounds__(kThreads) void tree_accept_kernel(AcceptParams p) {
  const int lane = threadIdx.x & 63;
  const int b = int(blockIdx.x) * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (b >= p.tree.batch) return;
  const Nodes s = nodes_of(p.tree, b);
  const int32_t* const parents = p.tree.parents + s.lo;
  const int32_t* const drafted = p.drafted + s.lo;
  const int32_t* const sampled = p.sampled + s.lo;
  int32_t* const path = p.path + long(b) * p.path_ld;
  // the first 64 nodes stay in registers
  int parent0 = -1, drafted0 = -1, sampled0 = -1;
  if (lane < s.n) {
    parent0 = parents[lane];
    drafted0 = drafted[lane];
    sampled0 = sampled[lane];
  }
  int count = 0, node = -1, token = -1;
  if (s.n > 0) {
    node = 0;
    count = 1;
    token = __builtin_amdgcn_readlane(sampled0, 0);
    if (lane == 0) path[0] = 0;
  }
  while (count > 0 && count < p.max_path && token >= 0) {
    int found = -1;
    for (int base = (node + 1) & ~63; base < s.n; base += 64) {
      const int at = base + lane;
      int parent = parent0, text = drafted0;
      if (base > 0 && at < s.n) {
        parent = parents[at];
        text = drafted[at];
      }
      const uint64_t hit = __ballot(at > node && at < s.n && parent == node && text == token);
      if (hit) {
        found = base + __builtin_ctzll(hit);
        break;
      }
    }
    if (found < 0) break;
    node = found;
    token = node < 64 ? __builtin_amdgcn_readlane(sampled0, node) : sampled[node];
    if (lane == 0) path[count] = node;
    ++count;
  }
  for (int i = count + lane; i < p.max_path; i += 64) path[i] = -1;
  if (lane == 0) {
    p.count[b] = count;
    p.tokens[b] = token;
    p.new_lens[b] = p.tree.lens[b] - s.n + count;
  }
}

// One wave a sequence, keys or values, and kv head; it takes the pages that get
// tokens in turn, so that a later page's codes and scale are still what they were
// when an earlier one takes tokens from it.  Within a page tokens move to
// lower slots in ascending order, so none is overwritten before it is read.
__global__ __launch_bounds__(kThreads) void kv_keep_kernel(KeepParams p, int units) {
  const KvArgs& kv = p.kv;
  const int lane = threadIdx.x & 63;
  const int unit = int(blockIdx.x) * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (unit >= units) return;
  const int head = unit % kv.kv_heads;
  const int which = unit / kv.kv_heads & 1;
  const int b = unit / (2 * kv.kv_heads);
  const kv::Seq s = kv::seq_of(kv, b);
  const int n = s.hi - s.lo, start = kv::told_length(kv, b) - n;
  const int count = min(min(p.count[b], p.max_path), n);
  if (count <= 0 || start < 0) return;
  const int32_t* const path = p.path + long(b) * p.path_ld;
  const long block_at = (long(which * kv.kv_heads + head) << kv.page_shift) * kv.dim;
  const long scale_at = which * kv.kv_heads + head;
  const int slot_mask = (1 << kv.page_shift) - 1;
  const int per = kv.dim >> 4;                    // lanes of a token
  const int together = 64 / per;                  // tokens at once
  const int group = lane / per, chunk = lane - group * per;

  // the page of the token that goes to place i, or -1
  auto source = [&](int i, int* node) {
    *node = path[i];
    return *node >= i && *node < n ? kv::page_at(kv, b, (start + *node) >> kv.page_shift) : -1;
  };
  auto scale_of = [&](int page) { return uint32_t(kv.scale[page * kv.scale_stride + scale_at]) & 0x7FFFu; };

  const int last = min((start + count - 1) >> kv.page_shift, kv.max_pages - 1);
  for (int index = start >> kv.page_shift; index <= last; ++index) {
    const int begin = index << kv.page_shift;
    const int i0 = max(begin - start, 0), i1 = min(begin + slot_mask + 1 - start, count);
    const int held = max(start - begin, 0);       // slots with earlier tokens
    const int page = kv::page_at(kv, b, index);
    if (page < 0) continue;
    const uint32_t was = scale_of(page);
    uint32_t bits = held > 0 ? was : 0u;
    bool any = false;
    for (int i = i0 + lane; i < i1; i += 64) {
      int node;
      const int from = source(i, &node);
      if (from >= 0) {
        bits = max(bits, scale_of(from));
        any = true;
      }
    }
    if (!__ballot(any)) continue;
    bits = wave_max_u32(bits);
    const float now = h2f(uint16_t(bits));
    int8_t* const block = kv.data + page * kv.page_stride + block_at;
    if (held > 0 && bits != was) {
      const float ratio = h2f(uint16_t(was)) / now;
      for (int i = lane; i < held * per; i += 64) {
        uint4* at = reinterpret_cast<uint4*>(block + long(i) * 16);
        uint4 w = *at;
        w.x = kv::rescale4(w.x, ratio);
        w.y = kv::rescale4(w.y, ratio);
        w.z = kv::rescale4(w.z, ratio);
        w.w = kv::rescale4(w.w, ratio);
        *at = w;
      }
    }
    for (int i = i0; i < i1; i += together) {
      const int to = i + group;
      int node = -1, from = -1;
      uint4 w = {0, 0, 0, 0};
      float ratio = 1.0f;
      if (group < together && to < i1) {
        from = source(to, &node);
        if (from >= 0) {
          const uint32_t old = from == page ? was : scale_of(from);
          if (old != bits) ratio = h2f(uint16_t(old)) / now;
          w = *reinterpret_cast<const uint4*>(kv.data + from * kv.page_stride + block_at +
                                              long((start + node) & slot_mask) * kv.dim + chunk * 16);
        }
      }
      // a token that stays where it is under the same scale is not written
      if (from >= 0 && (node != to || ratio != 1.0f)) {
        if (ratio != 1.0f) {
          w.x = kv::rescale4(w.x, ratio);
          w.y = kv::rescale4(w.y, ratio);
          w.z = kv::rescale4(w.z, ratio);
          w.w = kv::rescale4(w.w, ratio);
        }
        *reinterpret_cast<uint4*>(block + long((start + to) & slot_mask) * kv.dim + chunk * 16) = w;
      }
    }
    if (lane == 0 && bits != was) kv.scale[page * kv.scale_stride + scale_at] = uint16_t(bits);
  }
}

}  // namespace

hipError_t launch_tree_mask(const TreeMaskParams& p, hipStream_t stream) {
  TreeMaskParams a = p;
  void* args[] = {&a};
  return hipLaunchKernel(reinterpret_cast<const void*>(&tree_mask_kernel),
                         dim3(unsigned((p.tree.total_q + kThreads - 1) / kThreads)), dim3(kThreads), args, 0,
                         stream);
}

hipError_t launch_tree_accept(const AcceptParams& p, hipStream_t stream) {
  AcceptParams a = p;
  void* args[] = {&a};
  return hipLaunchKernel(reinterpret_cast<const void*>(&tree_accept_kernel),
                         dim3(unsigned((p.tree.batch + 3) / 4)), dim3(kThreads), args, 0, stream);
}

hipError_t launch_kv_keep(const KeepParams& p, hipStream_t stream) {
  KeepParams a = p;
  int units = p.kv.batch * 2 * p.kv.kv_heads;
  void* args[] = {&a, &units};
  return hipLaunchKernel(reinterpret_cast<const void*>(&kv_keep_kernel), dim3(unsigned((units + 3) / 4)),
                         dim3(kThreads), args, 0, stream);
}

}  // namespace w4a8
