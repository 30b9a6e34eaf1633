// sdpa_paged.cuh -- what the two forms of the paged attention share: their
// arguments, a sequence's extent, and the loading of key/value tiles page by
// page.
#pragma once

#include <atomic>

#include "internal.h"
#include "kv_pages.cuh"
#include "ptx_cluster.cuh"

namespace mha {

struct PagedSdpaArgs {
  const void* Q;
  int64_t q_stride;  // elements from token to token
  PagesView pages;
  const int32_t* q_offsets;
  void* O;  // [T, H, d]
  int T, H, G, max_new;
  bool causal, out_f32;
  float scale;
  int splits;  // 0: choose
  cudaStream_t stream;
};

constexpr int kPagedMaxSplits = 16;
constexpr int kPagedFewRows = 16;  // query slots of the few-rows form

cudaError_t launch_sdpa_paged_few(const PagedSdpaArgs& a, const DeviceCtl& ctl);
cudaError_t launch_sdpa_paged_rows(const PagedSdpaArgs& a, const DeviceCtl& ctl);

// Kernel arguments.
struct PagedParams {
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* q_offsets;
  void* O;
  int B, cols, num_pages, page_shift, kv_heads;
  int T, H, G, max_new, causal, out_f32, splits;
  float scale_log2;  // scale * log2(e)
  float inv_G;       // 1 / G
  unsigned* err;
  uint64_t limit_ns;
};

// x / G for 0 <= x < 512: the quotient's fraction is a multiple of 1/G, and
// half a unit of G keeps the product away from whole numbers by at least
// 1/256, far above its rounding (a division takes about 35 instructions).
__device__ __forceinline__ int div_by_group(const PagedParams& p, int x) {
  return static_cast<int>((static_cast<float>(x) + 0.5f) * p.inv_G);
}

inline PagedParams paged_params(const PagedSdpaArgs& a, const DeviceCtl& ctl) {
  return PagedParams{a.pages.table, a.pages.kv_len, a.q_offsets, a.O, a.pages.B, a.pages.cols,
                     a.pages.num_pages, a.pages.page_shift, a.pages.kv_heads, a.T, a.H, a.G,
                     a.max_new, a.causal, a.out_f32, a.splits,
                     static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634),
                     1.f / static_cast<float>(a.G), ctl.err, ctl.limit_ns};
}

// The tensor maps of Q [T, H, d], of `tokens` tokens and one group of heads
// per box, and of one layer's pools [P, Hkv * page, d], boxes of `rows` rows
// that stay inside a page.
inline bool paged_tensor_maps(const PagedSdpaArgs& a, int d, int tokens, int tile_rows,
                              CUtensorMap* q, CUtensorMap* k, CUtensorMap* v) {
  const uint64_t u2 = 2;
  const uint64_t qd[3] = {static_cast<uint64_t>(d), static_cast<uint64_t>(a.H),
                          static_cast<uint64_t>(a.T)};
  const uint64_t qs[2] = {d * u2, static_cast<uint64_t>(a.q_stride) * 2};
  const uint32_t qb[3] = {64, static_cast<uint32_t>(a.G), static_cast<uint32_t>(tokens)};
  const int page = 1 << a.pages.page_shift;
  const uint64_t pd[3] = {static_cast<uint64_t>(d),
                          static_cast<uint64_t>(a.pages.kv_heads) << a.pages.page_shift,
                          static_cast<uint64_t>(a.pages.num_pages)};
  const uint64_t pst[2] = {d * u2, static_cast<uint64_t>(a.pages.page_stride) * 2};
  const uint32_t pb[3] = {64, static_cast<uint32_t>(page < tile_rows ? page : tile_rows), 1};
  return encode_tensor_map(q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.Q), qd, qs,
                           qb, CU_TENSOR_MAP_SWIZZLE_128B) &&
         encode_tensor_map(k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.pages.K, pd, pst, pb,
                           CU_TENSOR_MAP_SWIZZLE_128B) &&
         encode_tensor_map(v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.pages.V, pd, pst, pb,
                           CU_TENSOR_MAP_SWIZZLE_128B);
}

// Sequence b's new tokens [q0, q0 + n) and length; bad: its length, its
// offsets (then n = 0).
struct PagedSeq {
  int q0, n, len;
  bool bad_len, bad_offsets;
};

__device__ __forceinline__ PagedSeq paged_seq_of(const PagedParams& p, int q0, int q1, int len) {
  PagedSeq s{};
  s.len = len;
  s.bad_offsets = q0 < 0 || q1 < q0 || q1 > p.T || q1 - q0 > p.max_new;
  s.q0 = q0;
  s.n = s.bad_offsets ? 0 : q1 - q0;
  const int64_t cap = static_cast<int64_t>(p.cols) << p.page_shift;
  s.bad_len = s.n > 0 && (s.len < 1 || s.len > cap || (p.causal && s.len < s.n));
  return s;
}

__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int b) {
  return paged_seq_of(p, __ldg(p.q_offsets + b), __ldg(p.q_offsets + b + 1), __ldg(p.kv_len + b));
}

// The page boxes of one tile of ROWS keys, one per lane of the producer warp:
// lane = page of the tile * KB + 64-column block.
template <int ROWS, int KB>
struct PageBoxes {
  int page;   // this lane's page number
  bool mine;  // this lane has a box of the tile

  // Request the page number of the tile that starts at key `key0`.
  __device__ __forceinline__ void fetch(const PagedParams& p, int b, int key0, int len, int lane) {
    const int slot = lane / KB;
    const int in_tile = ROWS >> p.page_shift;  // 0: the tile is part of a page
    const int entry = (key0 >> p.page_shift) + slot;
    mine = slot < (in_tile > 0 ? in_tile : 1) &&
           (static_cast<int64_t>(entry) << p.page_shift) < len;
    page = 0;
    if (mine) page = __ldg(p.table + static_cast<int64_t>(b) * p.cols + entry);
  }
  __device__ __forceinline__ bool in_range(const PagedParams& p) const {
    return static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages);
  }
  // The box is to be loaded, or its page number is out of range.
  __device__ __forceinline__ bool good(const PagedParams& p) const { return mine && in_range(p); }
  __device__ __forceinline__ bool bad(const PagedParams& p) const { return mine && !in_range(p); }
  // Bytes that the warp's boxes bring (warp-collective).
  __device__ __forceinline__ uint32_t bytes(const PagedParams& p) const {
    const uint32_t rows = min(ROWS, 1 << p.page_shift);
    return __popc(__ballot_sync(0xffffffffu, good(p))) * rows * 128u;
  }
  // Load this lane's box of head g into the tile at `dst` ([KB][ROWS][128 B]).
  __device__ __forceinline__ void load(const PagedParams& p, const CUtensorMap* map, uint32_t dst,
                                       uint32_t bar, int key0, int g, int lane) const {
    if (!good(p)) return;
    const int slot = lane / KB, kb = lane % KB;
    const int row = (key0 & ((1 << p.page_shift) - 1)) + (g << p.page_shift);
    tma_load_3d(dst + kb * (ROWS * 128) + (slot << p.page_shift) * 128, map, bar, kb * 64, row,
                page);
  }
};

// Store four consecutive outputs (fp32 or bf16) at element `at`.
__device__ __forceinline__ void store_out4(const PagedParams& p, int64_t at, float4 o) {
  if (p.out_f32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p.O) + at) = o;
  } else {
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.O) + at) =
        make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
  }
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t caddr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(caddr)
               : "memory");
  return v;
}

// The merge of a cluster's splits runs once per CTA, on code that no earlier
// instruction has brought near: its loops stay rolled, since fetching unrolled
// ones took longer (9 us at sixteen splits) than the remote loads, about a
// thousand clocks each, that they kept under way.

// Whether any CTA of the cluster met a bad page number (warp-collective; flag
// at the same shared address in every CTA).
__device__ __forceinline__ bool any_bad(uint32_t flag_at, int splits) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  if (lane < splits)
    bad = __float_as_uint(ld_cluster_f32(cluster_map(flag_at, static_cast<uint32_t>(lane)))) != 0u;
  return __any_sync(0xffffffffu, bad);
}

// One split's weight of a row, 2^(m_s - max m) / sum, from the row's maxima
// and sums of all splits (s * stride apart).  0 where no split saw a key (the
// sum is 0); a NaN among the scores has made the sum NaN and reaches the
// output.
__device__ __forceinline__ float split_weight(const float* m, const float* l, int stride,
                                              int splits, int s) {
  float top = -INFINITY, sum = 0.f;
#pragma unroll 1
  for (int k = 0; k < splits; ++k) top = fmaxf(top, m[k * stride]);
  if (top == -INFINITY) top = 0.f;
#pragma unroll 1
  for (int k = 0; k < splits; ++k) sum = fmaf(ex2_approx(m[k * stride] - top), l[k * stride], sum);
  return sum == 0.f ? 0.f : ex2_approx(m[s * stride] - top) / sum;
}

// o += weight * partial output at `from` in split s.  A weight of 0 stands for
// nothing seen, and for rows to be zeroed, whose partial output may be
// anything.
__device__ __forceinline__ void add_split(float4& o, uint32_t from, int s, float weight) {
  const float4 v = ld_cluster_f32x4(cluster_map(from, static_cast<uint32_t>(s)));
  if (weight != 0.f) {
    o.x = fmaf(weight, v.x, o.x);
    o.y = fmaf(weight, v.y, o.y);
    o.z = fmaf(weight, v.z, o.z);
    o.w = fmaf(weight, v.w, o.w);
  }
}

// Threads that share one place of the merged output: a power of two, as many
// as there are splits for and threads to spare.
__device__ __forceinline__ int merge_sharers(int places, int splits, int threads) {
  int n = 1;
  while (n < 16 && 2 * n <= splits && 2 * n * places <= threads) n *= 2;
  return n;
}

// Sum over the `sharers` neighbouring threads of a place, in a fixed order.
__device__ __forceinline__ void sum_sharers(float4& o, int sharers) {
#pragma unroll 1
  for (int k = 1; k < sharers; k *= 2) {
    o.x += __shfl_xor_sync(0xffffffffu, o.x, k);
    o.y += __shfl_xor_sync(0xffffffffu, o.y, k);
    o.z += __shfl_xor_sync(0xffffffffu, o.z, k);
    o.w += __shfl_xor_sync(0xffffffffu, o.w, k);
  }
}

// Bounded wait that ignores the abort flag (copies and products in flight).
__device__ __forceinline__ void paged_wait_drain(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > limit_ns) return;
  }
}

// Let a kernel use `smem_bytes` of shared memory, all of the unified array for
// it, and clusters of up to 16: set once per device and kernel (`done` holds a
// bit per device; above 64 devices it is set every time).
cudaError_t paged_kernel_attributes(const void* kernel, int smem_bytes,
                                    std::atomic<uint64_t>* done);

// Clusters of `splits` CTAs of a kernel with this block size and shared
// memory that the device holds at once (0 when it cannot be asked).
int paged_resident_clusters(int threads, int smem_bytes, int splits);

// Split count for `blocks` blocks over sequences of up to `capacity` keys.
int paged_default_splits(int64_t blocks, int64_t capacity, int threads, int smem_bytes);

}  // namespace mha
