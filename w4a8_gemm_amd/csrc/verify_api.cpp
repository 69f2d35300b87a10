// C ABI entry points of the operators that verify and end a decoding step:
// argument validation (host only, before any HIP call) and launch plans.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/w4a8.h"
#include "decoder_checks.h"
#include "decoder_kernels.h"
#include "verify_kernels.h"

using namespace w4a8;

namespace {

constexpr long kIntMax = 2147483647l;

// What tree_attention launches for a batch: row tiles of 16 a workgroup, and the
// workgroups that share each kv head's work.
struct TreePlan {
  int tiles, groups, shares, least, unit;
  size_t ml_bytes, workspace;
};

constexpr long kResident = 512;          // workgroups: two a compute unit
constexpr int kLeastSteps = 16;
constexpr long kMuchWork = 65536;

TreePlan plan_tree(const KvArgs& kv, int q_heads, int max_q, int max_len) {
  TreePlan pl;
  const int group = q_heads / kv.kv_heads;
  const long rows = long(kv.cu_q ? max_q : 1) * group;
  const long steps = (long(max_len) + kTreeStep - 1) / kTreeStep;
  // 32 rows a workgroup share the conversion of the codes, 16 leave more
  // workgroups and less to do before and after the keys.  By the products of 16
  // rows and a step there are, us with 16 rows and with 32, heads of 128: 3500 (one
  // tree of 26 tokens over 2001 keys) 13.8 and 16.5; 11000 20.6 and 21.3; 17000 27.6
  // and 25.1; 33000 (2 trees of 64) 35 and 28.7, (8 of 40) 27.6 and 30.5; 51000 52
  // and 42; 72000 66 and 53; 111000 74 and 53; 128000 (one of 64 over 30000) 121 and
  // 68; 169000 (16 of up to 64 over 4096) 89 and 73.  Heads of 64: 43000 (6 of up to
  // 200 over 1700) 20 and 24; 46000 27.2 and 31.4; 77000 33.9 and 37.9.  One limit
  // for both: below it heads of 128 lose up to a quarter, above it heads of 64 up to
  // an eighth.  64 rows take too many registers for more than two waves a SIMD and
  // measured 27, 33, 82 and 72 on the trees of 3500, 43000 and 169000 products and
  // on 4 of 13 over 50000 (16 rows 86, 32 75).
  const long products = attn_tiles(kv, group, 16) * kv.kv_heads * steps;
  pl.tiles = rows <= 16 || products < kMuchWork ? 1 : 2;
  // Tiles are split where they do not fill the device and there are keys for
  // two parts of kLeastSteps (one tree over 2001 keys: parts of 8 steps 16.9 us, of
  // 16 13.8).  Three workgroups a unit measured 77 against 73 us on the 16 trees,
  // 75 and 75 on the long ones.  The host knows how many tiles there may be, not how
  // long each is: where they may fill the device none is split, and a long sequence
  // among many short ones is one workgroup's a head (64 of 8 nodes, one of them over
  // 50000 keys, 420 us, and 13.6 with that one over 100).
  const long tiles = attn_tiles(kv, group, 16 * pl.tiles);
  pl.least = kLeastSteps;
  pl.shares = int(std::max(kResident / kv.kv_heads, tiles));
  if (steps < 2 * kLeastSteps || kResident / kv.kv_heads <= tiles || kv.batch > kTreeBatch) pl.shares = 0;
  pl.groups = int(pl.shares ? long(pl.shares) : tiles);
  const long longest = (long(kv.max_pages) << kv.page_shift) / kTreeStep + 1;
  for (pl.unit = 0; tiles * ((longest >> pl.unit) + 1) > kMostWork && pl.unit < 26; ++pl.unit) {
  }
  const size_t parts = pl.shares ? size_t(pl.groups) * kv.kv_heads * 16 * pl.tiles : 0;
  pl.ml_bytes = parts * 8;
  pl.workspace = pl.ml_bytes + parts * size_t(kv.dim) * 4;
  return pl;
}

// A batch of drafted tokens.
w4a8_status check_tree(const int32_t* parents, const int32_t* lens, const int32_t* cu_q, int batch,
                       int total_q, TreeBatch* t) {
  if (batch < 0 || total_q < 0 || batch > W4A8_M_MAX || total_q > W4A8_M_MAX)
    return W4A8_ERR_INVALID_ARGUMENT;
  if (!cu_q && total_q != batch) return W4A8_ERR_INVALID_ARGUMENT;
  if (batch > 0 && !lens) return W4A8_ERR_INVALID_ARGUMENT;
  if (batch > 0 && total_q > 0 && !parents) return W4A8_ERR_INVALID_ARGUMENT;
  t->parents = parents;
  t->lens = lens;
  t->cu_q = cu_q;
  t->batch = batch;
  t->total_q = total_q;
  return W4A8_OK;
}

// Rows from which on sampling looks at them in several workgroups before it draws.
// Measured with and without, fp16, us, without filters, with top_k 50 and with
// top_p 0.9: 16384 logits, one row 16 and 17, 17 and 16, 30 and 20; 512 rows 30 and
// 27, 24 and 21, 59 and 31.  24576 logits, one row 16 and 22, 17 and 19, 30 and 25;
// 512 rows 35 and 35, 25 and 24, 71 and 71.  32768 logits, one row 16 and 27, 17
// and 21, 30 and 30; 512 rows 40 and 44, 27 and 28, 79 and 112.
constexpr int kLongRow = 24576;

// log2 of a page size, or -1
int page_shift_of(int page_size) {
  for (int shift = 4; shift <= 10; ++shift)
    if (page_size == 1 << shift) return shift;
  return -1;
}

// A table over a pool of pages, and where its successor goes.
w4a8_status check_table(const int32_t* table, int table_ld, int max_pages, int batch, int new_batch,
                        const int32_t* refs, int num_pages, int32_t* new_table, int new_ld,
                        int32_t* new_refs, TableArgs* t) {
  if (max_pages < 1 || batch < 0 || new_batch < 0 || num_pages < 1 || table_ld < max_pages ||
      new_ld < max_pages || batch > W4A8_M_MAX || new_batch > W4A8_M_MAX)
    return W4A8_ERR_INVALID_ARGUMENT;
  if (!refs || !new_refs || refs == new_refs) return W4A8_ERR_INVALID_ARGUMENT;
  if ((batch > 0 && !table) || (new_batch > 0 && !new_table) || (batch > 0 && table == new_table))
    return W4A8_ERR_INVALID_ARGUMENT;
  if (num_pages > kPageBlock * kPageBlocks) return W4A8_ERR_UNSUPPORTED;
  if (long(std::max(batch, new_batch)) * max_pages > kIntMax) return W4A8_ERR_UNSUPPORTED;
  t->table = table;
  t->table_ld = table_ld;
  t->max_pages = max_pages;
  t->batch = batch;
  t->refs = refs;
  t->num_pages = num_pages;
  t->new_table = new_table;
  t->new_ld = new_ld;
  t->new_refs = new_refs;
  return W4A8_OK;
}

}  // namespace

extern "C" w4a8_status w4a8_tree_mask(const int32_t* parents_dev, const int32_t* seq_lens_dev,
                                      const int32_t* cu_q_dev, int batch, int total_q,
                                      uint32_t* mask_dev, int mask_ld, int mask_words,
                                      int32_t* positions_dev, void* stream) {
  TreeMaskParams p;
  const w4a8_status st = check_tree(parents_dev, seq_lens_dev, cu_q_dev, batch, total_q, &p.tree);
  if (st != W4A8_OK) return st;
  if (mask_words < 1 || mask_ld < mask_words) return W4A8_ERR_INVALID_ARGUMENT;
  if (batch == 0 || total_q == 0) return W4A8_OK;
  if (!mask_dev) return W4A8_ERR_INVALID_ARGUMENT;
  p.mask = mask_dev;
  p.mask_ld = mask_ld;
  p.words = mask_words;
  p.positions = positions_dev;
  return device_status(launch_tree_mask(p, static_cast<hipStream_t>(stream)));
}

extern "C" size_t w4a8_tree_attention_workspace_size(const w4a8_kv_view* view, int q_heads, int max_q,
                                                     int max_len) {
  KvArgs kv;
  if (check_view(view, &kv) != W4A8_OK || view->batch == 0 || view->total_q == 0) return 0;
  if (check_heads(kv, q_heads) != W4A8_OK || max_q < 0 || max_len < 0) return 0;
  return plan_tree(kv, q_heads, max_q, max_len).workspace;
}

extern "C" w4a8_status w4a8_tree_attention(const uint16_t* q_dev, int ldq, int q_heads,
                                           const w4a8_kv_view* view, const uint32_t* mask_dev,
                                           int mask_ld, int mask_words, int max_q, int max_len,
                                           float scale, int window, uint16_t* out_dev, int ldo,
                                           void* workspace_dev, size_t workspace_bytes, void* stream) {
  TreeAttnParams p;
  w4a8_status st = check_view(view, &p.kv);
  if (st != W4A8_OK) return st;
  if (max_q < 0 || max_len < 0 || window < 0 || !std::isfinite(scale) || mask_words < 1 ||
      mask_ld < mask_words)
    return W4A8_ERR_INVALID_ARGUMENT;
  if (view->batch == 0 || view->total_q == 0) return W4A8_OK;
  st = check_heads(p.kv, q_heads);
  if (st != W4A8_OK) return st;
  const long cols = long(q_heads) * p.kv.dim;
  if (!mask_dev || !rows_ok(q_dev, ldq, cols) || !rows_ok(out_dev, ldo, cols))
    return W4A8_ERR_INVALID_ARGUMENT;
  const TreePlan pl = plan_tree(p.kv, q_heads, max_q, max_len);
  if (long(pl.groups) * p.kv.kv_heads > kMaxWgs256) return W4A8_ERR_UNSUPPORTED;
  if (pl.workspace > 0) {
    if (workspace_bytes < pl.workspace) return W4A8_ERR_BUFFER_TOO_SMALL;
    if (!workspace_dev || !aligned16(workspace_dev)) return W4A8_ERR_INVALID_ARGUMENT;
  }
  p.q = q_dev;
  p.out = out_dev;
  p.ldq = ldq;
  p.ldo = ldo;
  p.q_heads = q_heads;
  p.group = q_heads / p.kv.kv_heads;
  p.scale_log2e = scale * 1.44269504f;
  p.window = window;
  p.tiles = pl.tiles;
  p.groups = pl.groups;
  p.shares = pl.shares;
  p.least = pl.least;
  p.unit = pl.unit;
  p.part_ml = static_cast<float2*>(workspace_dev);
  p.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace_dev) + (pl.workspace ? pl.ml_bytes : 0));
  p.mask = mask_dev;
  p.mask_ld = mask_ld;
  p.mask_words = mask_words;
  p.group_inverse = p.group > 1 ? uint32_t(((1ull << 32) + p.group - 1) / p.group) : 0u;
  return device_status(launch_tree_attn(p, static_cast<hipStream_t>(stream)));
}

extern "C" w4a8_status w4a8_tree_accept(const int32_t* drafted_dev, const int32_t* parents_dev,
                                        const int32_t* sampled_dev, const int32_t* seq_lens_dev,
                                        const int32_t* cu_q_dev, int batch, int total_q,
                                        int32_t* path_dev, int path_ld, int max_path,
                                        int32_t* count_dev, int32_t* tokens_dev,
                                        int32_t* new_lens_dev, void* stream) {
  AcceptParams p;
  const w4a8_status st = check_tree(parents_dev, seq_lens_dev, cu_q_dev, batch, total_q, &p.tree);
  if (st != W4A8_OK) return st;
  if (max_path < 1 || path_ld < max_path) return W4A8_ERR_INVALID_ARGUMENT;
  if (batch == 0) return W4A8_OK;
  if ((total_q > 0 && (!drafted_dev || !sampled_dev)) || !path_dev || !count_dev || !tokens_dev ||
      !new_lens_dev)
    return W4A8_ERR_INVALID_ARGUMENT;
  p.drafted = drafted_dev;
  p.sampled = sampled_dev;
  p.path = path_dev;
  p.path_ld = path_ld;
  p.max_path = max_path;
  p.count = count_dev;
  p.tokens = tokens_dev;
  p.new_lens = new_lens_dev;
  return device_status(launch_tree_accept(p, static_cast<hipStream_t>(stream)));
}

extern "C" w4a8_status w4a8_kv_keep(const w4a8_kv_view* view, const int32_t* path_dev, int path_ld,
                                    int max_path, const int32_t* count_dev, void* stream) {
  KeepParams p;
  const w4a8_status st = check_view(view, &p.kv);
  if (st != W4A8_OK) return st;
  if (max_path < 1 || path_ld < max_path) return W4A8_ERR_INVALID_ARGUMENT;
  if (view->batch == 0 || view->total_q == 0) return W4A8_OK;
  if (!path_dev || !count_dev) return W4A8_ERR_INVALID_ARGUMENT;
  if (2l * view->batch * view->kv_heads > 4 * kMaxWgs256) return W4A8_ERR_UNSUPPORTED;
  p.path = path_dev;
  p.path_ld = path_ld;
  p.max_path = max_path;
  p.count = count_dev;
  return device_status(launch_kv_keep(p, static_cast<hipStream_t>(stream)));
}

namespace {

// Whether a call asks its rows before it draws, and the workspace for it.
struct SamplePlan {
  int blocks, groups, parts;
  size_t masses_at, bins_at, list_at, maxima_at, listed_at, workspace;      // tops first
};

SamplePlan plan_sample(int logits_f32, int rows, int vocab) {
  SamplePlan pl = {};
  if (vocab < kLongRow) return pl;
  const int each = logits_f32 ? 4 : 8;
  const long chunks = (long(vocab) + each - 2) / each + 1;      // wherever the row begins
  pl.blocks = int((chunks + kSampleSpan - 1) / kSampleSpan);
  pl.groups = int((chunks + kSampleGroup - 1) / kSampleGroup);
  pl.parts = int((chunks + 63) / 64);
  if (long(rows) * pl.blocks > kMaxWgs256) return SamplePlan{};
  pl.masses_at = size_t(rows) * pl.blocks * 8;
  pl.bins_at = pl.masses_at + size_t(rows) * pl.parts * 8;
  pl.list_at = pl.bins_at + size_t(rows) * kSampleBins * 8;
  pl.maxima_at = pl.list_at + size_t(rows) * kSampleList * 8;
  pl.listed_at = pl.maxima_at + size_t(rows) * pl.groups * 4;
  pl.workspace = pl.listed_at + size_t(rows) * 4;
  return pl;
}

bool sample_sizes_ok(int rows, int vocab) {
  return rows >= 0 && rows <= W4A8_M_MAX && vocab >= 1 && vocab <= W4A8_VOCAB_MAX;
}

}  // namespace

extern "C" size_t w4a8_sample_workspace_size(int logits_f32, int rows, int vocab) {
  return sample_sizes_ok(rows, vocab) ? plan_sample(logits_f32, rows, vocab).workspace : 0;
}

extern "C" w4a8_status w4a8_sample(const void* logits_dev, int logits_f32, int ld, int rows, int vocab,
                                   const float* u_dev, const w4a8_sampling* settings,
                                   int32_t* tokens_dev, float* probs_dev, void* workspace_dev,
                                   size_t workspace_bytes, void* stream) {
  if (rows < 0 || rows > W4A8_M_MAX || vocab < 1 || ld < vocab || !settings)
    return W4A8_ERR_INVALID_ARGUMENT;
  if (vocab > W4A8_VOCAB_MAX) return W4A8_ERR_UNSUPPORTED;
  const w4a8_sampling& s = *settings;
  if ((!s.temperature_dev && !(s.temperature >= 0.0f && std::isfinite(s.temperature))) ||
      (!s.top_p_dev && std::isnan(s.top_p)) || (!s.min_p_dev && std::isnan(s.min_p)))
    return W4A8_ERR_INVALID_ARGUMENT;
  if (rows == 0) return W4A8_OK;
  if (!logits_dev || !u_dev || !tokens_dev) return W4A8_ERR_INVALID_ARGUMENT;
  if (reinterpret_cast<uintptr_t>(logits_dev) % (logits_f32 ? 4 : 2)) return W4A8_ERR_INVALID_ARGUMENT;
  const SamplePlan pl = plan_sample(logits_f32, rows, vocab);
  if (workspace_bytes < pl.workspace) return W4A8_ERR_BUFFER_TOO_SMALL;
  if (pl.workspace > 0 && (!workspace_dev || !aligned16(workspace_dev))) return W4A8_ERR_INVALID_ARGUMENT;
  SampleParams p;
  p.logits = logits_dev;
  p.f32 = logits_f32;
  p.ld = ld;
  p.rows = rows;
  p.vocab = vocab;
  p.u = u_dev;
  p.s = s;
  p.tokens = tokens_dev;
  p.probs = probs_dev;
  p.blocks = pl.blocks;
  p.groups = pl.groups;
  p.parts = pl.parts;
  // no row's weights are all wanted if every row has a top_k, or only a min_p
  const bool counts = !s.top_k_dev && s.top_k > 0 && s.top_k < vocab;
  const bool only_least = !s.top_p_dev && s.top_p >= 1.0f && !s.min_p_dev && s.min_p > 0.0f;
  const bool greedy = !s.temperature_dev && s.temperature == 0.0f;
  p.sums = !counts && !only_least && !greedy;
  const bool shares = p.sums && (s.top_p_dev || s.top_p < 1.0f);
  char* const ws = static_cast<char*>(workspace_dev);
  p.tops = pl.workspace ? reinterpret_cast<uint64_t*>(ws) : nullptr;
  p.masses = pl.workspace ? reinterpret_cast<uint64_t*>(ws + pl.masses_at) : nullptr;
  p.bins = pl.workspace && shares ? reinterpret_cast<uint64_t*>(ws + pl.bins_at) : nullptr;
  p.list = pl.workspace ? reinterpret_cast<uint2*>(ws + pl.list_at) : nullptr;
  p.maxima = pl.workspace ? reinterpret_cast<uint32_t*>(ws + pl.maxima_at) : nullptr;
  p.listed = pl.workspace ? reinterpret_cast<int32_t*>(ws + pl.listed_at) : nullptr;
  return device_status(launch_sample(p, static_cast<hipStream_t>(stream)));
}

extern "C" w4a8_status w4a8_kv_fork(const int32_t* block_table_dev, int block_table_ld, int max_pages,
                                    const int32_t* seq_lens_dev, int batch, const int32_t* refs_dev,
                                    int num_pages, int page_size, const int32_t* parent_dev,
                                    int new_batch, int32_t* new_table_dev, int new_table_ld,
                                    int32_t* new_lens_dev, int32_t* new_refs_dev, void* stream) {
  ForkParams p;
  const w4a8_status st = check_table(block_table_dev, block_table_ld, max_pages, batch, new_batch, refs_dev,
                                     num_pages, new_table_dev, new_table_ld, new_refs_dev, &p.t);
  if (st != W4A8_OK) return st;
  p.page_shift = page_shift_of(page_size);
  if (p.page_shift < 0) return W4A8_ERR_UNSUPPORTED;
  if (long(max_pages) << p.page_shift > kIntMax - page_size) return W4A8_ERR_INVALID_ARGUMENT;
  if ((batch > 0 && !seq_lens_dev) || (new_batch > 0 && (!parent_dev || !new_lens_dev)) ||
      (new_batch > 0 && seq_lens_dev == new_lens_dev))
    return W4A8_ERR_INVALID_ARGUMENT;
  p.lens = seq_lens_dev;
  p.parent = parent_dev;
  p.new_batch = new_batch;
  p.new_lens = new_lens_dev;
  return device_status(launch_kv_fork(p, static_cast<hipStream_t>(stream)));
}

extern "C" size_t w4a8_kv_alloc_workspace_size(int batch, int num_pages) {
  if (batch < 0 || batch > W4A8_M_MAX || num_pages < 1 || num_pages > kPageBlock * kPageBlocks) return 0;
  return (2 * size_t(num_pages) + size_t(page_blocks(num_pages)) + 5 * size_t(batch)) * 4;
}

extern "C" w4a8_status w4a8_kv_alloc(const int32_t* block_table_dev, int block_table_ld, int max_pages,
                                     const int32_t* seq_lens_dev, int batch, const int32_t* refs_dev,
                                     int num_pages, int page_size, const int32_t* tokens_dev, int tokens,
                                     int32_t* new_table_dev, int new_table_ld, int32_t* new_lens_dev,
                                     int32_t* new_refs_dev, int32_t* src_dev, int32_t* dst_dev,
                                     int32_t* counts_dev, void* workspace_dev, size_t workspace_bytes,
                                     void* stream) {
  AllocParams p;
  const w4a8_status st = check_table(block_table_dev, block_table_ld, max_pages, batch, batch, refs_dev,
                                     num_pages, new_table_dev, new_table_ld, new_refs_dev, &p.t);
  if (st != W4A8_OK) return st;
  p.page_shift = page_shift_of(page_size);
  if (p.page_shift < 0) return W4A8_ERR_UNSUPPORTED;
  if (long(max_pages) << p.page_shift > kIntMax - page_size || tokens < 0) return W4A8_ERR_INVALID_ARGUMENT;
  if (!counts_dev || (batch > 0 && (!seq_lens_dev || !new_lens_dev || !src_dev || !dst_dev ||
                                    seq_lens_dev == new_lens_dev)))
    return W4A8_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < w4a8_kv_alloc_workspace_size(batch, num_pages)) return W4A8_ERR_BUFFER_TOO_SMALL;
  if (!workspace_dev || !aligned16(workspace_dev)) return W4A8_ERR_INVALID_ARGUMENT;
  p.lens = seq_lens_dev;
  p.tokens_dev = tokens_dev;
  p.tokens = tokens;
  p.new_lens = new_lens_dev;
  p.src = src_dev;
  p.dst = dst_dev;
  p.counts = counts_dev;
  p.writers = static_cast<int32_t*>(workspace_dev);
  p.final_row = p.writers + num_pages;
  p.block_free = p.final_row + num_pages;
  p.row_need = p.block_free + page_blocks(num_pages);
  p.row_base = p.row_need + batch;
  p.row_held = p.row_base + batch;
  p.row_pair = p.row_held + batch;
  p.row_over = p.row_pair + batch;
  return device_status(launch_kv_alloc(p, static_cast<hipStream_t>(stream)));
}

extern "C" size_t w4a8_kv_compact_workspace_size(int num_pages) {
  if (num_pages < 1 || num_pages > kPageBlock * kPageBlocks) return 0;
  return (size_t(num_pages) + size_t(page_blocks(num_pages))) * 4;
}

extern "C" w4a8_status w4a8_kv_compact(const int32_t* block_table_dev, int block_table_ld, int max_pages,
                                       int batch, const int32_t* refs_dev, int num_pages,
                                       int32_t* new_table_dev, int new_table_ld, int32_t* new_refs_dev,
                                       int32_t* place_dev, int32_t* src_dev, int32_t* dst_dev,
                                       int32_t* counts_dev, void* workspace_dev, size_t workspace_bytes,
                                       void* stream) {
  CompactParams p;
  const w4a8_status st = check_table(block_table_dev, block_table_ld, max_pages, batch, batch, refs_dev,
                                     num_pages, new_table_dev, new_table_ld, new_refs_dev, &p.t);
  if (st != W4A8_OK) return st;
  if (!place_dev || !counts_dev || (num_pages > 1 && (!src_dev || !dst_dev)))
    return W4A8_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < w4a8_kv_compact_workspace_size(num_pages)) return W4A8_ERR_BUFFER_TOO_SMALL;
  if (!workspace_dev || !aligned16(workspace_dev)) return W4A8_ERR_INVALID_ARGUMENT;
  p.place = place_dev;
  p.src = src_dev;
  p.dst = dst_dev;
  p.counts = counts_dev;
  p.rank = static_cast<int32_t*>(workspace_dev);
  p.block_live = p.rank + num_pages;
  return device_status(launch_kv_compact(p, static_cast<hipStream_t>(stream)));
}

extern "C" w4a8_status w4a8_kv_copy_pages(int8_t* data_dev, uint16_t* scale_dev, long long page_stride,
                                          long long scale_stride, int num_pages, int page_size,
                                          int kv_heads, int head_dim, const int32_t* src_dev,
                                          const int32_t* dst_dev, int pairs, const int32_t* count_dev,
                                          void* stream) {
  if (num_pages < 1 || kv_heads < 1 || pairs < 0) return W4A8_ERR_INVALID_ARGUMENT;
  if (page_shift_of(page_size) < 0 || kv_heads > W4A8_HEADS_MAX || head_dim < 16 ||
      head_dim > W4A8_HEAD_DIM_MAX || head_dim % 16)
    return W4A8_ERR_UNSUPPORTED;
  const long bytes = 2l * kv_heads * page_size * head_dim;
  if (page_stride < bytes || page_stride % 16 || scale_stride < 2l * kv_heads)
    return W4A8_ERR_INVALID_ARGUMENT;
  if (bytes > 1l << 30) return W4A8_ERR_UNSUPPORTED;
  if (pairs == 0) return W4A8_OK;
  if (!data_dev || !scale_dev || !src_dev || !dst_dev || !aligned16(data_dev))
    return W4A8_ERR_INVALID_ARGUMENT;
  CopyParams p;
  p.data = data_dev;
  p.scale = scale_dev;
  p.page_stride = long(page_stride);
  p.scale_stride = long(scale_stride);
  p.num_pages = num_pages;
  p.page_bytes = int(bytes);
  p.scales = 2 * kv_heads;
  p.src = src_dev;
  p.dst = dst_dev;
  p.pairs = pairs;
  p.count = count_dev;
  return device_status(launch_kv_copy(p, static_cast<hipStream_t>(stream)));
}
