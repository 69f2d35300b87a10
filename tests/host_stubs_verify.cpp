// Stand-ins for the device side of the operators that verify and end a decoding
// step, for a host-only build of verify_api.cpp under AddressSanitizer and
// UndefinedBehaviorSanitizer.  A launch checks what the kernels assume of its
// parameters (grids and indices within their types) and reports no device.
#include <hip/hip_runtime_api.h>

#include <cstdlib>

#include "../w4a8_gemm_amd/csrc/verify_kernels.h"

namespace w4a8 {

namespace {
void need(bool ok) {
  if (!ok) abort();
}
void check(const KvArgs& kv) {
  need(kv.data && kv.scale && kv.table && kv.lens && kv.num_pages > 0 && kv.kv_heads > 0);
  need(kv.dim >= 16 && kv.dim <= 256 && kv.dim % 16 == 0 && kv.page_shift >= 4 && kv.page_shift <= 10);
  need(kv.batch > 0 && kv.total_q > 0 && (kv.cu_q || kv.total_q == kv.batch));
  need((long(kv.max_pages) << kv.page_shift) < (1l << 31));
}
void check(const TreeBatch& t) {
  need(t.lens && t.batch > 0 && t.total_q >= 0 && t.total_q <= (1 << 22) && (t.cu_q || t.total_q == t.batch));
}
void check(const TableArgs& t, int rows) {
  need(t.refs && t.new_refs && t.refs != t.new_refs && t.num_pages > 0 && t.num_pages <= kPageBlock * kPageBlocks);
  need(t.max_pages > 0 && t.table_ld >= t.max_pages && t.new_ld >= t.max_pages && (t.batch == 0 || t.table));
  need(rows == 0 || t.new_table);
  need(long(rows > t.batch ? rows : t.batch) * t.max_pages < (1l << 31));
  need(t.batch + page_blocks(t.num_pages) <= kMaxWgs256);
}
}  // namespace

w4a8_status device_status(hipError_t e) { return e == hipSuccess ? W4A8_OK : W4A8_ERR_DEVICE; }
hipError_t launch_tree_mask(const TreeMaskParams& p, hipStream_t) {
  check(p.tree);
  need(p.tree.parents && p.tree.total_q > 0 && p.mask && p.words >= 1 && p.mask_ld >= p.words);
  return hipErrorNoDevice;
}
hipError_t launch_tree_attn(const TreeAttnParams& p, hipStream_t) {
  check(p.kv);
  need(p.mask && p.mask_words >= 1 && p.mask_ld >= p.mask_words && (p.tiles == 1 || p.tiles == 2));
  need(p.group * p.kv.kv_heads == p.q_heads && (p.group == 1 || p.group_inverse > 0));
  const long tiles = attn_tiles(p.kv, p.group, 16 * p.tiles);
  need(p.groups >= tiles && long(p.groups) * p.kv.kv_heads <= kMaxWgs256);
  need(p.shares == 0 || (p.shares == p.groups && p.kv.batch <= kTreeBatch && p.least > 0 && p.part_ml && p.part_o));
  // work in its units, of the longest sequences the table holds, fits what a lane counts
  const long longest = (long(p.kv.max_pages) << p.kv.page_shift) / kTreeStep + 1;
  need(p.unit >= 0 && p.unit <= 26 && tiles * ((longest >> p.unit) + 1) <= kMostWork);
  return hipErrorNoDevice;
}
hipError_t launch_tree_accept(const AcceptParams& p, hipStream_t) {
  check(p.tree);
  need(p.path && p.max_path >= 1 && p.path_ld >= p.max_path && p.count && p.tokens && p.new_lens);
  need(p.tree.total_q == 0 || (p.tree.parents && p.drafted && p.sampled));
  return hipErrorNoDevice;
}
hipError_t launch_kv_keep(const KeepParams& p, hipStream_t) {
  check(p.kv);
  need(p.path && p.count && p.max_path >= 1 && p.path_ld >= p.max_path);
  need(2l * p.kv.batch * p.kv.kv_heads + 3 < (1l << 31));
  need((2l * p.kv.batch * p.kv.kv_heads + 3) / 4 <= kMaxWgs256);
  return hipErrorNoDevice;
}
hipError_t launch_sample(const SampleParams& p, hipStream_t) {
  need(p.logits && p.u && p.tokens && p.rows > 0 && p.rows <= (1 << 22) && p.vocab >= 1);
  need(p.vocab <= W4A8_VOCAB_MAX && p.ld >= p.vocab);
  if (p.maxima) {
    const long each = p.f32 ? 4 : 8, chunks = (p.vocab + each - 1 + each - 1) / each;   // the most a row has
    need(p.tops && p.masses && long(p.rows) * p.blocks <= kMaxWgs256);
    need(long(p.blocks) * kSampleSpan >= chunks && long(p.groups) * kSampleGroup >= chunks && p.parts * 64l >= chunks);
    // the parts of the workspace, one behind the other
    auto at = [&](const void* q) { return reinterpret_cast<const char*>(q) - reinterpret_cast<const char*>(p.tops); };
    const long rows = p.rows, list = at(p.list);
    need(at(p.masses) >= rows * p.blocks * 8 && list - at(p.masses) >= rows * p.parts * 8 + rows * kSampleBins * 8);
    need(!p.bins || (at(p.bins) - at(p.masses) >= rows * p.parts * 8 && list - at(p.bins) >= rows * kSampleBins * 8));
    need(at(p.maxima) - list >= rows * kSampleList * 8 && at(p.listed) - at(p.maxima) >= rows * p.groups * 4);
    need(size_t(at(p.listed) + rows * 4) <= w4a8_sample_workspace_size(p.f32, p.rows, p.vocab));
    need(p.sums || !p.bins);
  }
  return hipErrorNoDevice;
}
hipError_t launch_kv_fork(const ForkParams& p, hipStream_t) {
  check(p.t, p.new_batch);
  need((p.t.batch == 0 || p.lens) && (p.new_batch == 0 || (p.parent && p.new_lens && p.new_lens != p.lens)));
  need((long(p.t.max_pages) << p.page_shift) < (1l << 31));
  return hipErrorNoDevice;
}
hipError_t launch_kv_alloc(const AllocParams& p, hipStream_t) {
  check(p.t, p.t.batch);
  need(p.counts && p.writers && (p.t.batch == 0 || (p.lens && p.new_lens && p.src && p.dst)));
  need((long(p.t.max_pages) << p.page_shift) < (1l << 31) && p.tokens >= 0);
  const size_t used = (p.row_over + p.t.batch) - p.writers;
  need(used * 4 <= w4a8_kv_alloc_workspace_size(p.t.batch, p.t.num_pages));
  return hipErrorNoDevice;
}
hipError_t launch_kv_compact(const CompactParams& p, hipStream_t) {
  check(p.t, p.t.batch);
  need(p.place && p.counts && p.rank && (p.t.num_pages < 2 || (p.src && p.dst)));
  const size_t used = (p.block_live + page_blocks(p.t.num_pages)) - p.rank;
  need(used * 4 <= w4a8_kv_compact_workspace_size(p.t.num_pages));
  return hipErrorNoDevice;
}
hipError_t launch_kv_copy(const CopyParams& p, hipStream_t) {
  need(p.data && p.scale && p.src && p.dst && p.pairs > 0 && p.num_pages > 0);
  need(p.page_bytes > 0 && p.page_bytes % 16 == 0 && p.page_bytes <= 1 << 30 && p.page_stride >= p.page_bytes);
  need(p.scale_stride >= p.scales);
  return hipErrorNoDevice;
}

}  // namespace w4a8
