// A batch of sequences over a paged cache, as kernels see it.
#pragma once

#include "batch_clip.h"
#include "common.cuh"

namespace moex {

struct BatchView {
  const int32_t* cu_q;
  const int32_t* ctx_len;
  const int32_t* table;
  int64_t table_stride;
  int64_t page_stride, head_stride, row_stride;
  int n_seqs, n_tokens, table_width;
  int page_shift, n_pages;
  uint32_t* status;
};

inline BatchView batch_view(const moex_paged_kv* kv, const moex_batch* b, uint32_t* status) {
  BatchView v;
  v.cu_q = b->cu_q;
  v.ctx_len = b->ctx_len;
  v.table = b->page_table;
  v.table_stride = b->table_stride;
  v.page_stride = kv->page_stride;
  v.head_stride = kv->head_stride;
  v.row_stride = kv->row_stride;
  v.n_seqs = b->n_seqs;
  v.n_tokens = b->n_tokens;
  v.table_width = b->table_width;
  v.page_shift = 0;
  while ((1 << v.page_shift) < kv->page_size) ++v.page_shift;
  v.n_pages = static_cast<int>(kv->n_pages);
  v.status = status;
  return v;
}

// The tokens and length of sequence b (table_width pages are at most 2^30 positions by the host's check).
__device__ __forceinline__ SeqView seq_view(const BatchView& v, int b) {
  return clip_seq(v.cu_q[b], v.cu_q[b + 1], v.ctx_len[b], v.n_tokens, v.table_width << v.page_shift);
}

// Whether tokens in front of the first sequence or behind the last, as sequence
// b's offsets show it, belong to none.
__device__ __forceinline__ bool uncovered(const BatchView& v, int b) {
  return (b == 0 && v.cu_q[b] != 0) || (b + 1 == v.n_seqs && v.cu_q[b + 1] != v.n_tokens);
}

// The sequence that token `tok` belongs to, or -1.
__device__ __forceinline__ int seq_of_token(const BatchView& v, int tok) {
  int lo = 0, hi = v.n_seqs;  // the first b with cu_q[b + 1] > tok
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (v.cu_q[mid + 1] > tok)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo < v.n_seqs && v.cu_q[lo] <= tok ? lo : -1;
}

// The page that holds position `pos` of sequence b, or -1 (and the status bit)
// when the table names no page of the cache.  pos < table_width pages.
__device__ __forceinline__ int page_of(const BatchView& v, int b, int pos) {
  const int p = v.table[b * v.table_stride + (pos >> v.page_shift)];
  if (p >= 0 && p < v.n_pages) return p;
  flag_status(v.status, DEV_BAD_BATCH);
  return -1;
}

// Element offset of key head h, position pos, in the page `page`.
__device__ __forceinline__ int64_t kv_offset(const BatchView& v, int page, int h, int pos) {
  return page * v.page_stride + h * v.head_stride + (pos & ((1 << v.page_shift) - 1)) * v.row_stride;
}

}  // namespace moex
