// kv_pages.cu -- moving the pages of a paged key/value cache: forking
// sequences and compacting the held pages into other pools; and the checks of
// an mha_kv_pages that every entry point taking one applies.
//
// A fork shares the parent's full pages and copies the rows of its last,
// partly filled one, so two sequences never write to one page.  Compaction
// takes liveness from the page tables alone: a page is held when some
// sequence's table names it within that sequence's length.
//
// Both are copies, bound by HBM: every byte that has to move is read and
// written once.  Measured: 96 forks of 24 parents over eight layers, 400 MB
// moved, 47 us (parents' pages come from L2 again); 1,600 pages of four layers
// compacted, 3.2 GB moved, 474 us, 6.8 TB/s; small ones 3 and 4 us.
#include <stdint.h>

#include "internal.h"
#include "kv_pages.cuh"
#include "ptx_pdl.cuh"

namespace mha {

namespace {

mha_status check_pages(const mha_kv_pages* p) {
  if (!p || !p->K || !p->V) return MHA_ERR_INVALID_ARG;
  // without sequences there is no table to point to
  if (p->B > 0 && (!p->page_table || !p->kv_lengths)) return MHA_ERR_INVALID_ARG;
  if (p->num_pages < 1 || p->page_size < 1 || p->kv_heads < 1 || p->d < 1 || p->layers < 1 ||
      p->B < 0 || p->table_cols < 1)
    return MHA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(p->K) | reinterpret_cast<uintptr_t>(p->V)) & 15u)
    return MHA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(p->page_table) | reinterpret_cast<uintptr_t>(p->kv_lengths)) & 3u)
    return MHA_ERR_INVALID_ARG;
  if (p->page_size < 16 || p->page_size > 256 || (p->page_size & (p->page_size - 1)))
    return MHA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(p->table_cols) * p->page_size > (int64_t{1} << 30))
    return MHA_ERR_UNSUPPORTED;
  if ((static_cast<int64_t>(p->d) * bytes_of(p->dtype)) % 16) return MHA_ERR_UNSUPPORTED;
  const int64_t page = static_cast<int64_t>(p->kv_heads) * p->page_size * p->d;
  if (page > (int64_t{1} << 31)) return MHA_ERR_UNSUPPORTED;
  for (int64_t s : {p->page_stride, p->layer_stride})
    if (s < 0 || (s > 0 && s < page) || s % p->d) return MHA_ERR_INVALID_ARG;
  return MHA_OK;
}

}  // namespace

mha_status validate_pages(const mha_kv_pages* p) {
  if (p && p->dtype != MHA_BF16 && p->dtype != MHA_F32) return MHA_ERR_INVALID_ARG;
  return check_pages(p);
}

mha_status validate_pages_e4m3(const mha_kv_pages* p, const mha_kv_scales* s) {
  if (!p || p->dtype != MHA_E4M3 || !s || !s->K || !s->V) return MHA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(s->K) | reinterpret_cast<uintptr_t>(s->V)) & 3u)
    return MHA_ERR_INVALID_ARG;
  return check_pages(p);
}

mha_status validate_pages_shape(const mha_kv_pages* p) {
  if (p && p->dtype != MHA_BF16 && p->dtype != MHA_F32 && p->dtype != MHA_E4M3)
    return MHA_ERR_INVALID_ARG;
  return check_pages(p);
}

mha_status validate_pages_any(const mha_kv_pages* p, const mha_kv_scales* s) {
  if (p && p->dtype == MHA_E4M3) return validate_pages_e4m3(p, s);
  return s ? MHA_ERR_INVALID_ARG : validate_pages(p);
}

namespace {

constexpr int kThreads = 256;

// The pools of all layers, in 16-byte units.
struct Pools {
  uint4* K;
  uint4* V;
  int64_t page_stride, layer_stride;
  int num_pages;
  // of a cache in 8 bits, [layers, num_pages, kv_heads]; else nullptr
  float* k_scale;
  float* v_scale;
};

Pools pools_of(const mha_kv_pages& p, const mha_kv_scales* s) {
  const int es = bytes_of(p.dtype);
  const int64_t ps = p.page_stride ? p.page_stride
                                   : static_cast<int64_t>(p.kv_heads) * p.page_size * p.d;
  const int64_t ls = p.layer_stride ? p.layer_stride : ps * p.num_pages;
  return Pools{static_cast<uint4*>(p.K), static_cast<uint4*>(p.V), ps * es / 16, ls * es / 16,
               p.num_pages, s ? s->K : nullptr, s ? s->V : nullptr};
}

// Copy n 16-byte vectors with a block, four loads of a thread under way at a
// time (the compiler may not move a load over a store that could alias it).
__device__ __forceinline__ void block_copy(uint4* __restrict__ to, const uint4* __restrict__ from,
                                           int n) {
  constexpr int kAtOnce = 4;
  for (int v0 = threadIdx.x; v0 < n; v0 += kThreads * kAtOnce) {
    uint4 x[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      if (v0 + k * kThreads < n) x[k] = from[v0 + k * kThreads];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      if (v0 + k * kThreads < n) to[v0 + k * kThreads] = x[k];
  }
}

__global__ void __launch_bounds__(kThreads)
    kv_fork_kernel(const Pools pool, int32_t* __restrict__ table, int32_t* kv_len,
                   const int32_t* __restrict__ parents, const int32_t* __restrict__ children,
                   const int32_t* __restrict__ fresh, int n, int B, int cols, int page_shift,
                   int kv_heads, int row_vecs, int layers, unsigned* err) {
  const int i = blockIdx.x;
  const int par = parents[i], chi = children[i], fr = fresh[i];
  const int64_t cap = static_cast<int64_t>(cols) << page_shift;
  const int in_range = par >= 0 && par < B && chi >= 0 && chi < B;
  const int len = in_range ? kv_len[par] : -1;
  const int full = len >> page_shift, rem = len & ((1 << page_shift) - 1);
  bool ok = in_range && len >= 0 && len <= cap;
  int src = -1;
  if (ok && rem) {
    src = table[static_cast<int64_t>(par) * cols + full];
    ok = src >= 0 && src < pool.num_pages && fr >= 0 && fr < pool.num_pages;
  }
  // no other pair of this call may name the child, or the fresh page where
  // this one needs it: what the pairs read is then written by none of them
  bool clash = false;
  for (int j = threadIdx.x; j < n; j += kThreads) {
    if (parents[j] == chi || (j != i && children[j] == chi)) clash = true;
    if (rem && j != i && fresh[j] == fr) {
      const int pj = parents[j];
      if (pj >= 0 && pj < B && (kv_len[pj] & ((1 << page_shift) - 1))) clash = true;
    }
  }
  if (__syncthreads_or(clash)) ok = false;
  if (!ok) {
    if (blockIdx.y == 0 && threadIdx.x == 0) atomicOr(err, kErrPages);
    return;
  }
  if (blockIdx.y == 0) {
    const int32_t* from = table + static_cast<int64_t>(par) * cols;
    int32_t* to = table + static_cast<int64_t>(chi) * cols;
    for (int j = threadIdx.x; j < full; j += kThreads) to[j] = from[j];
    if (threadIdx.x == 0) {
      if (rem) to[full] = fr;
      kv_len[chi] = len;
    }
  }
  const int slabs = layers * 2 * kv_heads;  // (layer, K or V, head)
  const int slab_stride = row_vecs << page_shift;
  const int vecs = rem * row_vecs;
  for (int s = blockIdx.y; s < slabs; s += gridDim.y) {
    const int g = s % kv_heads, kv = (s / kv_heads) & 1, y = s / (2 * kv_heads);
    uint4* base = (kv ? pool.V : pool.K) + y * pool.layer_stride + static_cast<int64_t>(g) * slab_stride;
    block_copy(base + fr * pool.page_stride, base + src * pool.page_stride, vecs);
    if (pool.k_scale && rem && threadIdx.x == 0) {
      float* scale = (kv ? pool.v_scale : pool.k_scale) +
                     static_cast<int64_t>(y) * pool.num_pages * kv_heads + g;
      scale[static_cast<int64_t>(fr) * kv_heads] = scale[static_cast<int64_t>(src) * kv_heads];
    }
  }
}

// ------------------------------------------------------------------ compaction

constexpr int kRankThreads = 1024;

// Which pages some sequence holds (one bit each), the held pages before each
// word of 32, and their number.  One block: the bits are set in its shared
// memory, 128 KB for the 2^20 pages that a pool may have, so nothing has to
// be cleared beforehand and nothing but the result is written; a warp takes a
// sequence at a time.
__global__ void __launch_bounds__(kRankThreads)
    kv_rank_kernel(const int32_t* __restrict__ table, const int32_t* __restrict__ kv_len, int B,
                   int cols, int page_shift, int num_pages, unsigned* __restrict__ bits_out,
                   int32_t* __restrict__ rank, int32_t* __restrict__ n_live, int room,
                   unsigned* err) {
  extern __shared__ unsigned bits[];
  __shared__ int sums[32];
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int words = (num_pages + 31) / 32;
  for (int w = threadIdx.x; w < words; w += kRankThreads) bits[w] = 0u;
  __syncthreads();
  for (int b = warp; b < B; b += kRankThreads / 32) {
    const int len = kv_len[b];
    if (len < 0 || len > (static_cast<int64_t>(cols) << page_shift)) {
      if (lane == 0) atomicOr(err, kErrPages);
      continue;
    }
    const int held = (len + (1 << page_shift) - 1) >> page_shift;
    const int32_t* row = table + static_cast<int64_t>(b) * cols;
#pragma unroll 4
    for (int j = lane; j < held; j += 32) {
      const int page = __ldg(row + j);
      if (static_cast<unsigned>(page) < static_cast<unsigned>(num_pages))
        atomicOr(bits + (page >> 5), 1u << (page & 31));
      else
        atomicOr(err, kErrPages);
    }
  }
  __syncthreads();
  int base = 0;
  for (int w0 = 0; w0 < words; w0 += kRankThreads) {
    const int w = w0 + threadIdx.x;
    const unsigned word = w < words ? bits[w] : 0u;
    const int c = __popc(word);
    int incl = c;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, s);
      if (lane >= s) incl += up;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    // every warp sums up the warps before it, and all of them
    int up_to = sums[lane];
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, up_to, s);
      if (lane >= s) up_to += up;
    }
    const int before = warp ? __shfl_sync(0xffffffffu, up_to, warp - 1) : 0;
    if (w < words) {
      bits_out[w] = word;
      rank[w] = base + before + incl - c;
    }
    base += __shfl_sync(0xffffffffu, up_to, 31);
    __syncthreads();  // the sums have been read
  }
  if (threadIdx.x == 0) {
    *n_live = base;
    if (base > room) atomicOr(err, kErrPages);
  }
}

__device__ __forceinline__ int rank_of(const unsigned* bits, const int32_t* rank, int page) {
  return rank[page >> 5] + __popc(bits[page >> 5] & ((1u << (page & 31)) - 1u));
}

struct Renumber {
  const int32_t* table;
  const int32_t* kv_len;
  int B, cols, page_shift;
  int32_t* out;
  int out_cols;
};

// Copy the held pages, blockIdx.y picking the layer and K or V; the last
// blockIdx.y renumbers the page tables, a sequence per block at a time.
__global__ void __launch_bounds__(kThreads)
    kv_move_kernel(const Pools src, const Pools dst, const unsigned* __restrict__ bits,
                   const int32_t* __restrict__ rank, int page_vecs, int kv_heads,
                   const Renumber tables) {
  pdl_wait();
  if (blockIdx.y == gridDim.y - 1) {
    for (int b = blockIdx.x; b < tables.B; b += gridDim.x) {
      const int len = tables.kv_len[b];
      if (len < 0 || len > (static_cast<int64_t>(tables.cols) << tables.page_shift)) continue;
      const int held = (len + (1 << tables.page_shift) - 1) >> tables.page_shift;
      for (int j = threadIdx.x; j < held; j += kThreads) {
        const int page = tables.table[static_cast<int64_t>(b) * tables.cols + j];
        int r = -1;
        if (static_cast<unsigned>(page) < static_cast<unsigned>(src.num_pages))
          r = rank_of(bits, rank, page);
        tables.out[static_cast<int64_t>(b) * tables.out_cols + j] = r < dst.num_pages ? r : -1;
      }
    }
    return;
  }
  const int kv = blockIdx.y & 1, y = blockIdx.y >> 1;
  const uint4* from0 = (kv ? src.V : src.K) + y * src.layer_stride;
  uint4* to0 = (kv ? dst.V : dst.K) + y * dst.layer_stride;
  for (int page = blockIdx.x; page < src.num_pages; page += gridDim.x) {
    if (!((bits[page >> 5] >> (page & 31)) & 1u)) continue;
    const int r = rank_of(bits, rank, page);
    if (r >= dst.num_pages) continue;
    block_copy(to0 + r * dst.page_stride, from0 + page * src.page_stride, page_vecs);
    if (src.k_scale) {
      const float* from = (kv ? src.v_scale : src.k_scale) +
                          (static_cast<int64_t>(y) * src.num_pages + page) * kv_heads;
      float* to = (kv ? dst.v_scale : dst.k_scale) +
                  (static_cast<int64_t>(y) * dst.num_pages + r) * kv_heads;
      for (int g = threadIdx.x; g < kv_heads; g += kThreads) to[g] = from[g];
    }
  }
}

constexpr int kMaxPages = 1 << 20;

int num_sms() {
  int dev = 0, v = 0;
  if (cudaGetDevice(&dev) == cudaSuccess &&
      cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && v > 0)
    return v;
  return 1;
}

int words_of(int num_pages) { return (num_pages + 31) / 32; }

// The entry points' common part, after the checks of the pages and scales.
mha_status fork_pages(const mha_kv_pages* pages, const mha_kv_scales* scales,
                      const int32_t* parents, const int32_t* children, const int32_t* fresh, int n,
                      mha_stream stream) {
  if (n < 0 || n > pages->B) return MHA_ERR_INVALID_ARG;
  if (n == 0) return MHA_OK;
  for (const int32_t* p : {parents, children, fresh})
    if (!p || (reinterpret_cast<uintptr_t>(p) & 3u)) return MHA_ERR_INVALID_ARG;
  DeviceCtl ctl;
  if (!device_ctl(&ctl)) return MHA_ERR_CUDA;
  const int es = bytes_of(pages->dtype);
  const int64_t slabs = static_cast<int64_t>(pages->layers) * 2 * pages->kv_heads;
  // every block checks its pair against all others first: no more blocks than
  // keep the SMs full (about sixteen each)
  const int64_t want = (16 * static_cast<int64_t>(num_sms()) + n - 1) / n;
  const dim3 grid(n, static_cast<unsigned>(slabs < want ? slabs : want));
  kv_fork_kernel<<<grid, kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      pools_of(*pages, scales), pages->page_table, pages->kv_lengths, parents, children, fresh, n,
      pages->B, pages->table_cols, page_shift_of(pages->page_size), pages->kv_heads,
      pages->d * es / 16, pages->layers, ctl.err);
  return cudaGetLastError() == cudaSuccess ? MHA_OK : MHA_ERR_CUDA;
}

size_t compact_workspace_bytes(int num_pages) {
  if (num_pages < 1 || num_pages > kMaxPages) return 0;
  return static_cast<size_t>(words_of(num_pages)) * 8;  // bits, ranks
}

mha_status compact_pages(const mha_kv_pages* src, const mha_kv_scales* src_scales,
                         const mha_kv_pages* dst, const mha_kv_scales* dst_scales, int32_t* n_live,
                         void* workspace, size_t workspace_bytes, mha_stream stream) {
  mha_status st = validate_pages_any(src, src_scales);
  if (st != MHA_OK) return st;
  if (!dst) return MHA_ERR_INVALID_ARG;
  mha_kv_pages to = *dst;
  to.kv_lengths = src->kv_lengths;  // dst's own are not used
  st = validate_pages_any(&to, dst_scales);
  if (st != MHA_OK) return st;
  if (src_scales && (src_scales->K == dst_scales->K || src_scales->V == dst_scales->V ||
                     src_scales->K == dst_scales->V || src_scales->V == dst_scales->K))
    return MHA_ERR_INVALID_ARG;
  if (src->num_pages > kMaxPages) return MHA_ERR_UNSUPPORTED;
  if (dst->dtype != src->dtype || dst->page_size != src->page_size ||
      dst->kv_heads != src->kv_heads || dst->d != src->d || dst->layers != src->layers ||
      dst->B != src->B || dst->table_cols < src->table_cols)
    return MHA_ERR_INVALID_ARG;
  if (dst->K == src->K || dst->V == src->V || dst->K == src->V || dst->V == src->K ||
      (dst->page_table && dst->page_table == src->page_table))
    return MHA_ERR_INVALID_ARG;
  if (!n_live || (reinterpret_cast<uintptr_t>(n_live) & 3u) || !workspace ||
      (reinterpret_cast<uintptr_t>(workspace) & 15u) ||
      workspace_bytes < compact_workspace_bytes(src->num_pages))
    return MHA_ERR_INVALID_ARG;
  if (src->layers > 32767) return MHA_ERR_UNSUPPORTED;
  DeviceCtl ctl;
  if (!device_ctl(&ctl)) return MHA_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int words = words_of(src->num_pages);
  unsigned* bits = static_cast<unsigned*>(workspace);
  int32_t* rank = reinterpret_cast<int32_t*>(bits + words);
  const int shift = page_shift_of(src->page_size);
  const int es = bytes_of(src->dtype);
  const int page_vecs = src->kv_heads * src->page_size * (src->d * es / 16);
  cudaError_t e = cudaFuncSetAttribute(kv_rank_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kMaxPages / 8);
  if (e != cudaSuccess) return MHA_ERR_CUDA;
  kv_rank_kernel<<<1, kRankThreads, static_cast<size_t>(words) * 4, s>>>(
      src->page_table, src->kv_lengths, src->B, src->table_cols, shift, src->num_pages, bits, rank,
      n_live, dst->num_pages, ctl.err);
  // the copies' blocks are placed while the ranks are computed, and wait
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(src->num_pages < 2048 ? src->num_pages : 2048, src->layers * 2 + 1);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const Renumber tables{src->page_table, src->kv_lengths, src->B, src->table_cols, shift,
                        dst->page_table, dst->table_cols};
  e = cudaLaunchKernelEx(&cfg, kv_move_kernel, pools_of(*src, src_scales), pools_of(*dst, dst_scales),
                         static_cast<const unsigned*>(bits), static_cast<const int32_t*>(rank),
                         page_vecs, src->kv_heads, tables);
  if (e != cudaSuccess) return MHA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MHA_OK : MHA_ERR_CUDA;
}

}  // namespace
}  // namespace mha

using namespace mha;

extern "C" {

mha_status kv_pages_fork(const mha_kv_pages* pages, const int32_t* parents,
                         const int32_t* children, const int32_t* fresh, int n, mha_stream stream) {
  const mha_status st = validate_pages(pages);
  return st != MHA_OK ? st : fork_pages(pages, nullptr, parents, children, fresh, n, stream);
}

mha_status kv_pages_fork_e4m3(const mha_kv_pages* pages, const mha_kv_scales* scales,
                              const int32_t* parents, const int32_t* children,
                              const int32_t* fresh, int n, mha_stream stream) {
  const mha_status st = validate_pages_e4m3(pages, scales);
  return st != MHA_OK ? st : fork_pages(pages, scales, parents, children, fresh, n, stream);
}

size_t kv_pages_compact_workspace_bytes(int num_pages) {
  return compact_workspace_bytes(num_pages);
}

mha_status kv_pages_compact(const mha_kv_pages* src, const mha_kv_pages* dst, int32_t* n_live,
                            void* workspace, size_t workspace_bytes, mha_stream stream) {
  return compact_pages(src, nullptr, dst, nullptr, n_live, workspace, workspace_bytes, stream);
}

mha_status kv_pages_compact_e4m3(const mha_kv_pages* src, const mha_kv_scales* src_scales,
                                 const mha_kv_pages* dst, const mha_kv_scales* dst_scales,
                                 int32_t* n_live, void* workspace, size_t workspace_bytes,
                                 mha_stream stream) {
  if (!src_scales || !dst_scales) return MHA_ERR_INVALID_ARG;
  return compact_pages(src, src_scales, dst, dst_scales, n_live, workspace, workspace_bytes,
                       stream);
}

}  // extern "C"
