// Argument checks that the entry points over the paged cache share (host only,
// before any HIP call).
#pragma once
#include <cstdint>

#include "../../include/w4a8.h"
#include "decoder_kernels.h"

namespace w4a8 {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// rows of `cols` fp16 values read and written 16 bytes at a time
inline bool rows_ok(const void* p, int ld, long cols) {
  return p && aligned16(p) && ld >= cols && ld % 8 == 0;
}

// The view's sizes and pointers; on success fills `a`.  A view of an empty
// batch or of no new tokens is accepted with null pointers (`a` is then
// not used).
inline w4a8_status check_view(const w4a8_kv_view* v, KvArgs* a) {
  if (!v) return W4A8_ERR_INVALID_ARGUMENT;
  if (v->num_pages < 1 || v->kv_heads < 1 || v->batch < 0 || v->total_q < 0 || v->max_pages < 1 ||
      v->block_table_ld < v->max_pages || v->batch > W4A8_M_MAX || v->total_q > W4A8_M_MAX)
    return W4A8_ERR_INVALID_ARGUMENT;
  if (v->head_dim < 16 || v->head_dim > W4A8_HEAD_DIM_MAX || v->head_dim % 16 ||
      v->kv_heads > W4A8_HEADS_MAX)
    return W4A8_ERR_UNSUPPORTED;
  int shift = 4;
  while (shift < 10 && (1 << shift) < v->page_size) ++shift;
  if (v->page_size != 1 << shift) return W4A8_ERR_UNSUPPORTED;
  if (long(v->max_pages) << shift > 2147483647l - v->page_size) return W4A8_ERR_INVALID_ARGUMENT;
  // without cu_q every sequence brings one token
  if (!v->cu_q_dev && v->total_q != v->batch) return W4A8_ERR_INVALID_ARGUMENT;
  const long block = long(v->page_size) * v->head_dim;
  const long page = 2l * v->kv_heads * block;
  if (v->page_stride < page || v->page_stride % 16 || v->scale_stride < 2l * v->kv_heads)
    return W4A8_ERR_INVALID_ARGUMENT;
  if (v->batch == 0 || v->total_q == 0) return W4A8_OK;
  if (!v->data_dev || !v->scale_dev || !v->block_table_dev || !v->seq_lens_dev)
    return W4A8_ERR_INVALID_ARGUMENT;
  if (!aligned16(v->data_dev)) return W4A8_ERR_INVALID_ARGUMENT;
  a->data = v->data_dev;
  a->scale = v->scale_dev;
  a->page_stride = long(v->page_stride);
  a->scale_stride = long(v->scale_stride);
  a->num_pages = v->num_pages;
  a->kv_heads = v->kv_heads;
  a->dim = v->head_dim;
  a->page_shift = shift;
  a->table = v->block_table_dev;
  a->table_ld = v->block_table_ld;
  a->max_pages = v->max_pages;
  a->lens = v->seq_lens_dev;
  a->cu_q = v->cu_q_dev;
  a->batch = v->batch;
  a->total_q = v->total_q;
  return W4A8_OK;
}

inline w4a8_status check_heads(const KvArgs& kv, int q_heads) {
  if (q_heads < 1) return W4A8_ERR_INVALID_ARGUMENT;
  if (q_heads % kv.kv_heads || q_heads > W4A8_HEADS_MAX) return W4A8_ERR_UNSUPPORTED;
  if (long(kv.total_q) * q_heads > 2147483647l) return W4A8_ERR_UNSUPPORTED;
  return W4A8_OK;
}

}  // namespace w4a8
