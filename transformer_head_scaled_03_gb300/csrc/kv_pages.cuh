// kv_pages.cuh -- one layer of a paged key/value cache as the kernels see it,
// and the checks and look-ups they share.
#pragma once

#include <stdint.h>

#include "internal.h"
#include "ptx.cuh"

namespace mha {

// One layer's pools, by value.  Element strides.
struct PagesView {
  void* K;
  void* V;
  int num_pages, page_shift, kv_heads, d;
  int64_t page_stride;
  const int32_t* table;
  const int32_t* kv_len;
  int B, cols;
  // of a cache in 8 bits, [num_pages, kv_heads]; else nullptr
  float* k_scale;
  float* v_scale;
};

inline int bytes_of(mha_dtype t) { return t == MHA_E4M3 ? 1 : t == MHA_BF16 ? 2 : 4; }

// log2 of a page size that pages_view has accepted.
inline int page_shift_of(int page_size) {
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

// The layer's view of checked pages.
inline PagesView pages_view(const mha_kv_pages& p, int layer, const mha_kv_scales* s = nullptr) {
  const int64_t ps = p.page_stride ? p.page_stride
                                   : static_cast<int64_t>(p.kv_heads) * p.page_size * p.d;
  const int64_t ls = p.layer_stride ? p.layer_stride : ps * p.num_pages;
  const int64_t off = ls * layer * bytes_of(p.dtype);
  const int64_t scale_off = static_cast<int64_t>(p.num_pages) * p.kv_heads * layer;
  return PagesView{static_cast<char*>(p.K) + off, static_cast<char*>(p.V) + off, p.num_pages,
                   page_shift_of(p.page_size), p.kv_heads, p.d, ps, p.page_table, p.kv_lengths,
                   p.B, p.table_cols, s ? s->K + scale_off : nullptr,
                   s ? s->V + scale_off : nullptr};
}

// Which packed token belongs to which sequence: the number of sequences that
// end at or before token t.  The offsets ascend, so that is t's sequence (B
// for a token behind the last one); the loads of a warp are independent, one
// round of B/32 each, where a binary search would chain log2(B) of them.
// Every lane of a converged warp calls this with the same t.
__device__ __forceinline__ int sequence_of_token(const int32_t* q_offsets, int B, int t) {
  const int lane = threadIdx.x & 31;
  int ended = 0;
  for (int b = lane; b < B; b += 32) ended += __ldg(q_offsets + b + 1) <= t ? 1 : 0;
  return static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(ended)));
}

}  // namespace mha
