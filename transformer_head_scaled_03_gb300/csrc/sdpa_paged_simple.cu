// sdpa_paged_simple.cu -- paged attention over a cache in 8 bits, a warp per
// query row: the online softmax over its keys, a lane holding D / 32 columns.
#include <math.h>
#include <stdint.h>

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "sdpa_paged.cuh"

namespace mha {
namespace {

__device__ __forceinline__ float sum32(float v) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

template <int D>
__global__ void __launch_bounds__(128)
    sdpa_paged_simple_kernel(const __nv_bfloat16* Q, int64_t q_stride, const __nv_fp8_e4m3* K,
                             const __nv_fp8_e4m3* V, int64_t page_stride, const PagedParams p) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= p.T * p.H) return;
  const int t = row / p.H, h = row - t * p.H, g = h / p.G;
  int b = t;
  if (p.q_offsets) {
    b = sequence_of_token(p.q_offsets, p.B, t);
    if (b >= p.B) return;
  }
  const PagedSeq s = paged_seq(p, b);
  if (s.bad_offsets || s.bad_len) {
    if (lane == 0) atomicOr(p.err, kErrPages);
    if (s.bad_offsets) return;
  }
  if (s.n == 0 || t < s.q0) return;
  int len = s.bad_len ? 0 : p.causal ? min(s.len, s.len - s.n + (t - s.q0) + 1) : s.len;
  const int32_t* table = table_row(p, b, g);
  const int held = s.bad_len ? 0 : (len + (1 << p.page_shift) - 1) >> p.page_shift;
  for (int j = 0; j < held; ++j) {
    if (static_cast<unsigned>(__ldg(table + j)) < static_cast<unsigned>(p.num_pages)) continue;
    if (lane == 0) atomicOr(p.err, kErrPages);
    len = 0;
  }
  float q[N], o[N], m = -INFINITY, l = 0.f;
  for (int i = 0; i < N; ++i) {
    q[i] = __bfloat162float(Q[t * q_stride + static_cast<int64_t>(h) * D + lane * N + i]);
    o[i] = 0.f;
  }
  for (int j = 0; j < len; ++j) {
    const int page = __ldg(table + (j >> p.page_shift));
    const int64_t at = page * page_stride +
                       ((static_cast<int64_t>(g) << p.page_shift) + (j & ((1 << p.page_shift) - 1))) * D +
                       lane * N;
    const int64_t sc = static_cast<int64_t>(page) * p.kv_heads + g;
    float x = 0.f;
    for (int i = 0; i < N; ++i) x = fmaf(q[i], static_cast<float>(K[at + i]), x);
    x = sum32(x) * p.k_scale[sc] * p.scale_log2;
    const float top = fmaxf(m, x), keep = exp2f(m - top), w = exp2f(x - top);
    l = l * keep + w;
    for (int i = 0; i < N; ++i)
      o[i] = o[i] * keep + w * p.v_scale[sc] * static_cast<float>(V[at + i]);
    m = top;
  }
  for (int i = 0; i < N; ++i) {
    const float y = len > 0 ? o[i] / l : 0.f;
    const int64_t at = static_cast<int64_t>(row) * D + lane * N + i;
    if (p.out_f32)
      static_cast<float*>(p.O)[at] = y;
    else
      static_cast<__nv_bfloat16*>(p.O)[at] = __float2bfloat16_rn(y);
  }
}

}  // namespace

cudaError_t launch_sdpa_paged_simple(const PagedSdpaArgs& a, const DeviceCtl& ctl) {
  const int64_t rows = static_cast<int64_t>(a.T) * a.H;
  if (rows > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  auto go = [&](auto kern) {
    kern<<<static_cast<unsigned>((rows + 3) / 4), 128, 0, a.stream>>>(
        static_cast<const __nv_bfloat16*>(a.Q), a.q_stride,
        static_cast<const __nv_fp8_e4m3*>(a.pages.K), static_cast<const __nv_fp8_e4m3*>(a.pages.V),
        a.pages.page_stride, paged_params(a, ctl));
  };
  if (a.pages.d == 64)
    go(sdpa_paged_simple_kernel<64>);
  else
    go(sdpa_paged_simple_kernel<128>);
  return cudaGetLastError();
}

}  // namespace mha
