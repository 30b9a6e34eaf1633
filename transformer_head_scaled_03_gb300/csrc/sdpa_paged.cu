// sdpa_paged.cu -- attention of packed new tokens over a paged key/value
// cache (decoding, chunks of prompts, mixed).
#include <math.h>
#include <stdint.h>

#include <cuda_bf16.h>

#include "internal.h"
#include "kv_pages.cuh"

namespace mha {
namespace {

struct PagedParams {
  const __nv_bfloat16* Q;
  int64_t q_stride;
  PagesView pages;
  const int32_t* q_offsets;
  void* O;
  int out_f32;
  int T, H, G, max_new, causal;
  float scale_log2;
  unsigned* err;
};

// One warp per (token, head): online softmax over the visible keys.
template <int D>
__global__ void __launch_bounds__(256) sdpa_paged_simple_kernel(const PagedParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(p.T) * p.H) return;
  const PagesView& pg = p.pages;
  const int t = static_cast<int>(row / p.H), h = static_cast<int>(row % p.H);
  const int b = sequence_of_token(p.q_offsets, pg.B, t);
  if (b >= pg.B) return;
  const int q0 = __ldg(p.q_offsets + b), q1 = __ldg(p.q_offsets + b + 1), n = q1 - q0;
  if (q0 < 0 || t < q0 || t >= q1 || q1 > p.T || n > p.max_new) {
    if (lane == 0) atomicOr(p.err, kErrPages);
    return;
  }
  const int len = __ldg(pg.kv_len + b);
  const bool bad = len < 1 || len > (static_cast<int64_t>(pg.cols) << pg.page_shift) ||
                   (p.causal && len < n);
  const int seen = bad ? 0 : p.causal ? len - n + (t - q0) + 1 : len;
  bool bad_page = bad;
  constexpr int N = D / 32;
  float q[N], o[N];
  for (int i = 0; i < N; ++i) {
    q[i] = __bfloat162float(p.Q[t * p.q_stride + static_cast<int64_t>(h) * D + i * 32 + lane]);
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < seen; ++j) {
    const int page = __ldg(pg.table + static_cast<int64_t>(b) * pg.cols + (j >> pg.page_shift));
    if (page < 0 || page >= pg.num_pages) {
      bad_page = true;
      break;
    }
    const int64_t at = page * pg.page_stride +
                       ((static_cast<int64_t>(h / p.G) << pg.page_shift) +
                        (j & ((1 << pg.page_shift) - 1))) * D + lane;
    float s = 0.f;
    for (int i = 0; i < N; ++i)
      s = fmaf(q[i], __bfloat162float(static_cast<const __nv_bfloat16*>(pg.K)[at + i * 32]), s);
    for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s), al = exp2f(m - mn), w = exp2f(s - mn);
    l = fmaf(l, al, w);
    for (int i = 0; i < N; ++i)
      o[i] = fmaf(o[i], al,
                  w * __bfloat162float(static_cast<const __nv_bfloat16*>(pg.V)[at + i * 32]));
    m = mn;
  }
  if (bad_page && lane == 0) atomicOr(p.err, kErrPages);
  const float inv = bad_page || l == 0.f ? 0.f : 1.f / l;
  for (int i = 0; i < N; ++i) {
    const int64_t at = row * D + i * 32 + lane;
    const float v = inv == 0.f ? 0.f : o[i] * inv;
    if (p.out_f32)
      static_cast<float*>(p.O)[at] = v;
    else
      static_cast<__nv_bfloat16*>(p.O)[at] = __float2bfloat16_rn(v);
  }
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
  if (T < 0 || H < 1 || max_new < 1 || layer < 0 || layer >= pages->layers ||
      H % pages->kv_heads != 0)
    return MHA_ERR_INVALID_ARG;
  if (out_dtype != MHA_BF16 && out_dtype != MHA_F32) return MHA_ERR_INVALID_ARG;
  if (!(scale >= 0.f) || isinf(scale)) return MHA_ERR_INVALID_ARG;
  if (mask_kind != MHA_MASK_NONE && mask_kind != MHA_MASK_CAUSAL_BOTTOM_RIGHT)
    return MHA_ERR_INVALID_ARG;
  if (num_splits < 0 || num_splits > 16) return MHA_ERR_INVALID_ARG;
  const int d = pages->d, G = H / pages->kv_heads;
  if (q_token_stride == 0) q_token_stride = static_cast<int64_t>(H) * d;
  if (q_token_stride < static_cast<int64_t>(H) * d || q_token_stride % 8)
    return MHA_ERR_INVALID_ARG;
  if (pages->dtype != MHA_BF16 || (d != 64 && d != 128) || G > 128) return MHA_ERR_UNSUPPORTED;
  if (T == 0 || pages->B == 0) return MHA_OK;
  for (const void* p : {Q, static_cast<const void*>(O)})
    if (!p || (reinterpret_cast<uintptr_t>(p) & 15u)) return MHA_ERR_INVALID_ARG;
  if (O == Q || !q_offsets || (reinterpret_cast<uintptr_t>(q_offsets) & 3u))
    return MHA_ERR_INVALID_ARG;
  DeviceCtl ctl;
  if (!device_ctl(&ctl)) return MHA_ERR_CUDA;
  const float sc = scale == 0.f ? static_cast<float>(1.0 / sqrt(static_cast<double>(d))) : scale;
  PagedParams p{static_cast<const __nv_bfloat16*>(Q), q_token_stride, pages_view(*pages, layer),
                q_offsets, O, out_dtype == MHA_F32, T, H, G, max_new,
                mask_kind == MHA_MASK_CAUSAL_BOTTOM_RIGHT,
                static_cast<float>(static_cast<double>(sc) * 1.4426950408889634), ctl.err};
  const int64_t rows = static_cast<int64_t>(T) * H;
  if ((rows + 7) / 8 > 0x7fffffffLL) return MHA_ERR_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>((rows + 7) / 8);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d == 64)
    sdpa_paged_simple_kernel<64><<<grid, 256, 0, s>>>(p);
  else
    sdpa_paged_simple_kernel<128><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? MHA_OK : MHA_ERR_CUDA;
}

}  // extern "C"
