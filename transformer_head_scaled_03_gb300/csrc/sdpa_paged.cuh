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
  PagesView pages;   // with a table per token and kv head: B = T, kv_len a token's
  const int32_t* q_offsets;  // nullptr: "sequence" t is token t alone
  bool head_tables;  // the page table is [B, kv_heads, cols]
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
cudaError_t launch_sdpa_paged_few_e4m3(const PagedSdpaArgs& a, const DeviceCtl& ctl);
cudaError_t launch_sdpa_paged_rows_e4m3(const PagedSdpaArgs& a, const DeviceCtl& ctl);
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
  const float* k_scale;  // of a cache in 8 bits, [num_pages, kv_heads]
  const float* v_scale;
  int head_tables;       // the page table has a row for every kv head
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
                     1.f / static_cast<float>(a.G), ctl.err, ctl.limit_ns, a.pages.k_scale,
                     a.pages.v_scale, a.head_tables};
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

// The row of the page table that sequence b's kv head g reads.
__device__ __forceinline__ const int32_t* table_row(const PagedParams& p, int b, int g) {
  return p.table + (p.head_tables ? static_cast<int64_t>(b) * p.kv_heads + g : b) * p.cols;
}

// The tensor maps of one layer's pools in 8 bits [P, Hkv * page, d], boxes of
// `rows` whole rows that stay inside a page.
inline bool paged_tensor_maps_e4m3(const PagedSdpaArgs& a, int d, int tile_rows, CUtensorMap* k,
                                   CUtensorMap* v) {
  const int page = 1 << a.pages.page_shift;
  const uint64_t pd[3] = {static_cast<uint64_t>(d),
                          static_cast<uint64_t>(a.pages.kv_heads) << a.pages.page_shift,
                          static_cast<uint64_t>(a.pages.num_pages)};
  const uint64_t pst[2] = {static_cast<uint64_t>(d), static_cast<uint64_t>(a.pages.page_stride)};
  const uint32_t pb[3] = {static_cast<uint32_t>(d),
                          static_cast<uint32_t>(page < tile_rows ? page : tile_rows), 1};
  const CUtensorMapSwizzle swizzle =
      d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  return encode_tensor_map(k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.pages.K, pd, pst, pb, swizzle) &&
         encode_tensor_map(v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.pages.V, pd, pst, pb, swizzle);
}

// Sequence b's new tokens [q0, q0 + n) and length; bad: its length, its
// offsets (then n = 0).  Without offsets a sequence is one token, passed over
// when its length is 0.
struct PagedSeq {
  int q0, n, len;
  bool bad_len, bad_offsets;
};

__device__ __forceinline__ PagedSeq paged_seq_of(const PagedParams& p, int q0, int q1, int len) {
  PagedSeq s{};
  s.len = len;
  s.bad_offsets = q0 < 0 || q1 < q0 || q1 > p.T || q1 - q0 > p.max_new;
  s.q0 = q0;
  s.n = s.bad_offsets || (!p.q_offsets && len == 0) ? 0 : q1 - q0;
  const int64_t cap = static_cast<int64_t>(p.cols) << p.page_shift;
  s.bad_len = s.n > 0 && (s.len < 1 || s.len > cap || (p.causal && s.len < s.n));
  return s;
}

__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int b) {
  const int len = __ldg(p.kv_len + b);
  return p.q_offsets ? paged_seq_of(p, __ldg(p.q_offsets + b), __ldg(p.q_offsets + b + 1), len)
                     : paged_seq_of(p, b, b + 1, len);
}

// Where sequence i's tokens start.
__device__ __forceinline__ int paged_offset(const PagedParams& p, int i) {
  return p.q_offsets ? __ldg(p.q_offsets + i) : i;
}

// The page boxes of one tile of ROWS keys, one per lane of the producer warp:
// lane = page of the tile * KB + column block of kRowBytes (64 columns in
// bf16; in 8 bits the whole row).
template <int ROWS, int KB, int kRowBytes = 128>
struct PageBoxes {
  int page;   // this lane's page number
  bool mine;  // this lane has a box of the tile

  // Request the page number of the tile that starts at key `key0`, from the
  // sequence's row of the page table.
  __device__ __forceinline__ void fetch(const PagedParams& p, const int32_t* row, int key0, int len,
                                        int lane) {
    const int slot = lane / KB;
    const int in_tile = ROWS >> p.page_shift;  // 0: the tile is part of a page
    const int entry = (key0 >> p.page_shift) + slot;
    mine = slot < (in_tile > 0 ? in_tile : 1) &&
           (static_cast<int64_t>(entry) << p.page_shift) < len;
    page = 0;
    if (mine) page = __ldg(row + entry);
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
    return __popc(__ballot_sync(0xffffffffu, good(p))) * rows *
           static_cast<uint32_t>(kRowBytes);
  }
  // Load this lane's box of head g into the tile at `dst` ([KB][ROWS][128 B]).
  __device__ __forceinline__ void load(const PagedParams& p, const CUtensorMap* map, uint32_t dst,
                                       uint32_t bar, int key0, int g, int lane) const {
    if (!good(p)) return;
    const int slot = lane / KB, kb = lane % KB;
    const int row = (key0 & ((1 << p.page_shift) - 1)) + (g << p.page_shift);
    tma_load_3d(dst + kb * (ROWS * kRowBytes) + (slot << p.page_shift) * kRowBytes, map, bar,
                kb * 64, row, page);
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

// The four softmax warps of the few-rows kernels.
__device__ __forceinline__ void softmax_bar() {
  asm volatile("bar.sync 1, 128;" ::: "memory");
}

// What the merge of the few-rows kernels keeps in shared memory, fp32: this
// CTA's m and l of the 16 slots and its partial outputs [16][d], then every
// split's m and l and the weights, [16 splits][16] each.
constexpr int few_merge_bytes(int d) {
  return (2 * kPagedFewRows + kPagedFewRows * d + 3 * kPagedMaxSplits * kPagedFewRows) * 4;
}

// Merge the splits through distributed shared memory (warps 0-3, after a
// cluster barrier): every split's m and l are fetched, each thread works out
// weights, 2^(m_s - M) / sum, then the outputs, four columns a place, each
// another remote load.
template <int D>
__device__ __forceinline__ void few_merge(const PagedParams& p, const PagedSeq& seq, int g,
                                          int split, float* xm, volatile int* bad_page) {
  constexpr int kSlots = kPagedFewRows;
  float* xl = xm + kSlots;
  float* xo = xl + kSlots;
  float* xw = xo + kSlots * D;
  const int rows = seq.n * p.G;
  const int S = p.splits;
  float* lm = xw + kPagedMaxSplits * kSlots;
  float* ll = lm + kPagedMaxSplits * kSlots;
  const uint32_t xm_s = smem_u32(xm), xl_s = smem_u32(xl), xo_s = smem_u32(xo);
  const bool bad = any_bad(smem_u32(const_cast<int*>(bad_page)), S);
#pragma unroll 1
  for (int x = threadIdx.x; x < S * kSlots; x += 128) {
    const uint32_t q = x % kSlots, s = x / kSlots;
    lm[x] = ld_cluster_f32(cluster_map(xm_s + 4u * q, s));
    ll[x] = ld_cluster_f32(cluster_map(xl_s + 4u * q, s));
  }
  softmax_bar();
#pragma unroll 1
  for (int x = threadIdx.x; x < S * kSlots; x += 128)
    xw[x] = bad ? 0.f : split_weight(lm + x % kSlots, ll + x % kSlots, kSlots, S, x / kSlots);
  softmax_bar();
  const int total = rows * (D / 4);
  const int per = (total + S - 1) / S;
  const int e0 = split * per;
  const int e1 = min(total, e0 + per);
  const int sharers = merge_sharers(per, S, 128);
#pragma unroll 1
  for (int f0 = e0; f0 < e1; f0 += 128 / sharers) {
    const int e = f0 + static_cast<int>(threadIdx.x) / sharers;
    const int q = e / (D / 4);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (e < e1) {
#pragma unroll 2
      for (int s = threadIdx.x % sharers; s < S; s += sharers)
        add_split(o, xo_s + 16u * e, s, xw[s * kSlots + q]);
    }
    sum_sharers(o, sharers);
    if (e < e1 && threadIdx.x % sharers == 0) {
      const int i = div_by_group(p, q);
      const int64_t row = static_cast<int64_t>(seq.q0 + i) * p.H + g * p.G + (q - i * p.G);
      store_out4(p, row * D + (e - q * (D / 4)) * 4, o);
    }
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
// graded: the merge's cost grows with the splits (the few-rows forms over pages in
// 8 bits and over selected pages; the others, query tiles in 8 bits among them,
// keep the choices they were measured with).
int paged_default_splits(int64_t blocks, int64_t capacity, int threads, int smem_bytes,
                         bool graded = false);

}  // namespace mha
