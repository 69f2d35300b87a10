// Launch interface of the operators that verify and end a decoding step: the
// masks of drafted trees, the confirmed path and its keys and values, sampling,
// and the pages of a cache that several sequences share.  The C ABI layer is
// verify_api.cpp.
#pragma once
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "../../include/w4a8.h"
#include "decoder_kernels.h"

namespace w4a8 {

// A batch's drafted tokens: sequence b's are [cu_q[b], cu_q[b + 1]) (one each
// without cu_q), parents before children.
struct TreeBatch {
  const int32_t* parents;
  const int32_t* lens;
  const int32_t* cu_q;
  int batch, total_q;
};

struct TreeMaskParams {
  TreeBatch tree;
  uint32_t* mask;
  long mask_ld;
  int words;
  int32_t* positions;         // may be null
};
hipError_t launch_tree_mask(const TreeMaskParams& p, hipStream_t stream);

struct TreeAttnParams {
  KvArgs kv;
  const uint16_t* q;
  uint16_t* out;
  int ldq, ldo;
  int q_heads, group;         // group = q_heads / kv_heads
  uint32_t group_inverse;     // 2^32 / group, rounded up (group > 1)
  float scale_log2e;          // score scale * log2(e)
  int window;                 // 0: none
  const uint32_t* mask;       // bit j of a new token's row: it sees the sequence's new token j
  long mask_ld;
  int mask_words;
  int tiles;                  // rows of a workgroup, in tiles of 16: 1 or 2
  int groups;                 // workgroups of a kv head: for all row tiles, and for
  int shares;                 // about as many parts as this of all work; 0: tiles are not split
  int least;                  // steps of a part, at least
  int unit;                   // log2 of the steps in which work is counted
  float2* part_ml;            // split tiles: [groups][kv_heads][16 * tiles] maximum and sum of the
  float* part_o;              // rows of a workgroup's part, and their unnormalised values, [dim] each
};
constexpr int kTreeStep = 32;          // keys of a step
constexpr int kTreeBatch = 4096;       // most sequences whose tiles are split: 64 a lane
constexpr long kMostWork = (1l << 25) - 1;   // what a lane counts: 64 of them fit an int
hipError_t launch_tree_attn(const TreeAttnParams& p, hipStream_t stream);

struct AcceptParams {
  TreeBatch tree;
  const int32_t* drafted;
  const int32_t* sampled;
  int32_t* path;
  long path_ld;
  int max_path;
  int32_t* count;
  int32_t* tokens;
  int32_t* new_lens;
};
hipError_t launch_tree_accept(const AcceptParams& p, hipStream_t stream);

struct KeepParams {
  KvArgs kv;
  const int32_t* path;
  long path_ld;
  int max_path;
  const int32_t* count;
};
hipError_t launch_kv_keep(const KeepParams& p, hipStream_t stream);

struct SampleParams {
  const void* logits;
  int f32;                    // else fp16
  long ld;
  int rows, vocab;
  const float* u;
  w4a8_sampling s;
  int32_t* tokens;
  float* probs;               // may be null
  // long rows: what is known of them before (workspace; null: nothing)
  int blocks, groups, parts;  // of a row: workgroups, groups of chunks, stretches of 64 chunks
  bool sums;                  // some row may need sums of all its weights
  uint32_t* maxima;           // [rows][groups] largest keys
  uint64_t* tops;             // [rows][blocks] largest key, and bit 32: a logit is NaN or infinite
  uint64_t* masses;           // [rows][parts] sums of weights
  uint64_t* bins;             // [rows][kSampleBins] sums of weights; null: no row may need them
  uint2* list;                // [rows][kSampleList] tokens of one bin: key, place
  int32_t* listed;            // [rows] their number; more than kSampleList: not listed
};
constexpr int kSampleBins = 2048, kSampleList = 4096;
// Chunks of 16 bytes that a workgroup looks at before.  512, 1024 and 2048 measured,
// one row of 128256 fp16 logits 14, 16 and 21 us, with top_p 26, 29 and 39; 801 of
// 152064 with mixed filters 226, 210 and 231; 512 of 128256 with top_p 254, 189 and
// 177: sums in bins of each workgroup are added to the row's.
constexpr int kSampleSpan = 1024;
constexpr int kSampleGroup = 8;         // chunks of a group
hipError_t launch_sample(const SampleParams& p, hipStream_t stream);

// The pages of a pool, their reference counts and the tables that name them.
// Pages are counted in blocks of kPageBlock, at most kPageBlocks of them.
constexpr int kPageBlock = 1024;
constexpr int kPageBlocks = W4A8_PAGES_MAX / kPageBlock;
struct TableArgs {
  const int32_t* table;
  long table_ld;
  int max_pages, batch;
  const int32_t* refs;
  int num_pages;
  int32_t* new_table;
  long new_ld;
  int32_t* new_refs;
};

struct ForkParams {
  TableArgs t;
  const int32_t* lens;
  int page_shift;
  const int32_t* parent;
  int new_batch;
  int32_t* new_lens;
};
hipError_t launch_kv_fork(const ForkParams& p, hipStream_t stream);

struct AllocParams {
  TableArgs t;
  const int32_t* lens;
  int page_shift;
  const int32_t* tokens_dev;  // new tokens of each sequence; null: `tokens` each
  int tokens;
  int32_t* new_lens;
  int32_t* src;
  int32_t* dst;
  int32_t* counts;            // pairs of pages to copy, entries that got no page
  // workspace
  int32_t* writers;           // [num_pages]: sequences that write a shared page,
  int32_t* final_row;         // and the last of them
  int32_t* block_free;        // [blocks]: free pages, then those of the blocks before
  int32_t* row_need;          // [batch]: entries without a page that need one,
  int32_t* row_base;          // [batch]: requests of the sequences before,
  int32_t* row_held;          // [batch]: page to copy from, or -1,
  int32_t* row_pair;          // [batch]: its place among the pairs, or -1
  int32_t* row_over;          // [batch]: entries beyond the table
};
hipError_t launch_kv_alloc(const AllocParams& p, hipStream_t stream);

struct CompactParams {
  TableArgs t;
  int32_t* place;
  int32_t* src;
  int32_t* dst;
  int32_t* counts;
  int32_t* block_live;        // workspace, [blocks]: pages in use
  int32_t* rank;              // workspace, [num_pages]: place among the moved, or the filled, pages
};
hipError_t launch_kv_compact(const CompactParams& p, hipStream_t stream);

struct CopyParams {
  int8_t* data;
  uint16_t* scale;
  long page_stride, scale_stride;
  int num_pages;
  int page_bytes;             // a multiple of 16
  int scales;                 // of a page
  const int32_t* src;
  const int32_t* dst;
  int pairs;
  const int32_t* count;       // may be null: all pairs
};
hipError_t launch_kv_copy(const CopyParams& p, hipStream_t stream);

inline int page_blocks(int num_pages) { return (num_pages + kPageBlock - 1) / kPageBlock; }

}  // namespace w4a8
