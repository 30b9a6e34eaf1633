// sdpa_paged.cu -- the paged attention's entry point: argument checks, the
// choice of the kernel, and the split counts both kernels use.
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "sdpa_paged.cuh"

namespace mha {
namespace {

// Stand-in for the attention kernels in occupancy queries: a block of their
// size with their shared memory and no body (for kernels that allocate
// tensor memory the runtime's calculator answers one CTA per SM).
__global__ void paged_occupancy_proxy_kernel() {}

int max_active_clusters(int threads, int smem_bytes, int splits) {
  auto kern = paged_occupancy_proxy_kernel;
  int n = 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(splits));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem_bytes);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes) !=
          cudaSuccess ||
      cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                           cudaSharedmemCarveoutMaxShared) != cudaSuccess ||
      cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
          cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

}  // namespace

cudaError_t paged_kernel_attributes(const void* kernel, int smem_bytes,
                                    std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (done->load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
  return e;
}

int paged_resident_clusters(int threads, int smem_bytes, int splits) {
  // a cluster sits inside one GPC, so the device is asked for every size, once
  // per kernel
  struct Entry {
    int dev, threads, smem;
    int fits[kPagedMaxSplits + 1];
  };
  static std::mutex mutex;
  static Entry table[64];
  static int used = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lock(mutex);
  for (int i = 0; i < used; ++i)
    if (table[i].dev == dev && table[i].threads == threads && table[i].smem == smem_bytes)
      return table[i].fits[splits];
  Entry e{dev, threads, smem_bytes, {}};
  for (int s = 1; s <= kPagedMaxSplits; ++s) e.fits[s] = max_active_clusters(threads, smem_bytes, s);
  if (used < 64) table[used++] = e;
  return e.fits[splits];
}

int paged_default_splits(int64_t blocks, int64_t capacity, int threads, int smem_bytes,
                         bool graded) {
  // Time in units of one 128-key tile: a CTA's tiles, its set-up and first
  // loads (4), and the merge (3).  Waves of clusters: lengths differ and long
  // sequences go first, so a partial last wave costs something between its
  // share and a whole one.  Measured against every split count: within 5 % of
  // the best for one to 64 sequences of 200 to 32 K tokens, but for chunks of
  // very unequal sequences (20 tokens over 2 to 9 K keys: 94 us at the chosen
  // two, 86 at four).  The capacity stands for the lengths, which are on the
  // device: tables far wider than their sequences are split too often.  64
  // sequences of 200 to 1000 tokens take 45 us with room for 1 K or 32 K tokens
  // each and 80 us with room for 128 K; 16 of 16 to 32 K take 240 us with room
  // for 32 K as for 1 M.
  // Graded: one sequence of 2 K keys takes 16.4, 11.4, 9.0, 8.1 and 9.9 us on 1, 2,
  // 4, 8 and 16 CTAs per head, so a merge counts for about as many tiles as
  // the splits' binary logarithm and one, and for seven beyond eight CTAs (few
  // such clusters fit the GPCs).
  auto merge_of = [graded](int s) -> double {
    if (!graded) return s > 1 ? 3 : 0;
    return s == 1 ? 0 : s == 2 ? 1.8 : s <= 4 ? 2.7 : s <= 8 ? 3.7 : 7;
  };
  const double tiles = static_cast<double>(capacity) / 128;
  int best = 1;
  double least = 0;
  for (int s = 1; s <= kPagedMaxSplits && (s == 1 || s <= tiles); ++s) {
    const int fits = paged_resident_clusters(threads, smem_bytes, s);
    if (fits < 1) continue;
    const double waves = static_cast<double>(blocks) / fits;
    const double cost = (waves <= 1 ? 1 : 0.5 * (ceil(waves) + waves)) *
                        (tiles / s + 4 + merge_of(s));
    if (s == 1 || cost < least) {
      best = s;
      least = cost;
    }
  }
  return best;
}

namespace {

// The entry points' common part: the checks that follow those of the pages,
// and the choice of the kernel.  `selected`: a page table per token and kv
// head, [T, kv_heads, cols], with the tokens' lengths; else nullptr.
mha_status attend(const void* Q, int64_t q_token_stride, const mha_kv_pages* pages,
                  const mha_kv_scales* scales, int layer, const int32_t* q_offsets,
                  const int32_t* selected, const int32_t* lengths, int cols, void* O, int T, int H,
                  int max_new, float scale, int mask_kind, mha_dtype out_dtype, int num_splits,
                  mha_stream stream) {
  if (T < 0 || H < 1 || max_new < (T > 0 ? 1 : 0) || layer < 0 || layer >= pages->layers ||
      H % pages->kv_heads != 0)
    return MHA_ERR_INVALID_ARG;
  if (out_dtype != MHA_BF16 && out_dtype != MHA_F32) return MHA_ERR_INVALID_ARG;
  if (!(scale >= 0.f) || isinf(scale)) return MHA_ERR_INVALID_ARG;
  if (mask_kind != MHA_MASK_NONE && mask_kind != MHA_MASK_CAUSAL_BOTTOM_RIGHT)
    return MHA_ERR_INVALID_ARG;
  if (num_splits < 0 || num_splits > 16) return MHA_ERR_INVALID_ARG;
  const int d = pages->d, G = H / pages->kv_heads;
  if (q_token_stride == 0) q_token_stride = static_cast<int64_t>(H) * d;
  if (q_token_stride < static_cast<int64_t>(H) * d || q_token_stride % d)
    return MHA_ERR_INVALID_ARG;
  if (pages->dtype == MHA_F32 || (d != 64 && d != 128) || G > 128) return MHA_ERR_UNSUPPORTED;
  const bool by_token = !q_offsets && lengths;
  if (T == 0 || (!by_token && pages->B == 0)) return MHA_OK;
  for (const void* p : {Q, static_cast<const void*>(O)})
    if (!p || (reinterpret_cast<uintptr_t>(p) & 15u)) return MHA_ERR_INVALID_ARG;
  if (O == Q) return MHA_ERR_INVALID_ARG;
  if (by_token) {
    if (!selected || ((reinterpret_cast<uintptr_t>(selected) |
                       reinterpret_cast<uintptr_t>(lengths)) & 3u))
      return MHA_ERR_INVALID_ARG;
  } else if (!q_offsets || (reinterpret_cast<uintptr_t>(q_offsets) & 3u)) {
    return MHA_ERR_INVALID_ARG;
  }
  DeviceCtl ctl;
  if (!device_ctl(&ctl)) return MHA_ERR_CUDA;
  PagedSdpaArgs a;
  a.Q = Q;
  a.q_stride = q_token_stride;
  a.pages = pages_view(*pages, layer, scales);
  a.head_tables = by_token;
  if (by_token) {
    a.pages.table = selected;
    a.pages.kv_len = lengths;
    a.pages.B = T;
    a.pages.cols = cols;
  }
  a.q_offsets = q_offsets;
  a.O = O;
  a.T = T;
  a.H = H;
  a.G = G;
  a.max_new = max_new < T ? max_new : T;
  a.causal = mask_kind == MHA_MASK_CAUSAL_BOTTOM_RIGHT;
  a.out_f32 = out_dtype == MHA_F32;
  a.scale = scale == 0.f ? static_cast<float>(1.0 / sqrt(static_cast<double>(d))) : scale;
  a.splits = num_splits;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  // sixteen rows or fewer per kv head are the N side of the products, more
  // of them the M side.  One kernel takes all sequences: 63 single tokens over
  // 1 to 32 K keys beside a chunk of 512 over 32 K (32 heads on 8, d = 128) take
  // 856 us, where the single tokens alone take 667 and the chunk alone 229.
  // Single tokens with a loose max_new pay for it: 64 sequences of 200 to 1000
  // keys 59 us instead of 45, 16 of 16 to 32 K 279 instead of 240.
  const bool few = static_cast<int64_t>(a.max_new) * G <= kPagedFewRows;
  const cudaError_t e =
      few ? scales ? launch_sdpa_paged_few_e4m3(a, ctl) : launch_sdpa_paged_few(a, ctl)
      : scales ? launch_sdpa_paged_rows_e4m3(a, ctl)
               : launch_sdpa_paged_rows(a, ctl);
  return e == cudaSuccess ? MHA_OK : MHA_ERR_CUDA;
}

}  // namespace
}  // namespace mha

using namespace mha;

extern "C" {

mha_status sdpa_paged(const void* Q, int64_t q_token_stride, const mha_kv_pages* pages, int layer,
                      const int32_t* q_offsets, void* O, int T, int H, int max_new, float scale,
                      int mask_kind, mha_dtype out_dtype, int num_splits, mha_stream stream) {
  const mha_status st = validate_pages(pages);
  if (st != MHA_OK) return st;
  return attend(Q, q_token_stride, pages, nullptr, layer, q_offsets, nullptr, nullptr, 0, O, T, H,
                max_new, scale, mask_kind, out_dtype, num_splits, stream);
}

mha_status sdpa_paged_e4m3(const void* Q, int64_t q_token_stride, const mha_kv_pages* pages,
                           const mha_kv_scales* scales, int layer, const int32_t* q_offsets,
                           void* O, int T, int H, int max_new, float scale, int mask_kind,
                           mha_dtype out_dtype, int num_splits, mha_stream stream) {
  const mha_status st = validate_pages_e4m3(pages, scales);
  if (st != MHA_OK) return st;
  return attend(Q, q_token_stride, pages, scales, layer, q_offsets, nullptr, nullptr, 0, O, T, H,
                max_new, scale, mask_kind, out_dtype, num_splits, stream);
}

mha_status sdpa_paged_selected(const void* Q, int64_t q_token_stride, const mha_kv_pages* pages,
                               const mha_kv_scales* scales, int layer, const int32_t* selected,
                               const int32_t* lengths, int n_select, void* O, int T, int H,
                               float scale, mha_dtype out_dtype, int num_splits,
                               mha_stream stream) {
  const mha_status st = validate_pages_any(pages, scales);
  if (st != MHA_OK) return st;
  if (n_select < 1) return MHA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(n_select) * pages->page_size > (int64_t{1} << 30))
    return MHA_ERR_UNSUPPORTED;
  if (T > 0 && (!selected || !lengths)) return MHA_ERR_INVALID_ARG;
  return attend(Q, q_token_stride, pages, scales, layer, nullptr, selected, lengths, n_select, O, T,
                H, 1, scale, MHA_MASK_CAUSAL_BOTTOM_RIGHT, out_dtype, num_splits, stream);
}

}  // extern "C"
