// qk_norm_rope.cu -- the norm of every query and key head and the rotation by
// its position, in one pass; its gradient; and the serving form that appends
// the keys and values to a paged cache.
//
//   rstd = 1 / sqrt(mean(x^2) + eps),  xh = x * rstd,  z = xh * gamma
//   (y_a, y_b) = (z_a cos - z_b sin, z_b cos + z_a sin)  per pair of columns
// and backwards, with dz the rotation of dy by the opposite angle:
//   dgamma = sum over rows of dz * xh,  u = dz * gamma,
//   dx = rstd * (u - xh * mean(u * xh))
//
// About ten flops per element moved: bound by HBM, or by the launch when
// there are few rows.
#include <math.h>
#include <stdint.h>

#include <cuda_bf16.h>

#include "internal.h"
#include "kv_pages.cuh"

namespace mha {
namespace {

constexpr int kWarps = 8;
constexpr int kMaxD = 256;
constexpr int kMaxGradBlocks = 608;  // rows of dgamma partials

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// The columns of pair i.
__device__ __forceinline__ void pair_columns(int i, int r, int half, int* a, int* b) {
  *a = half ? i : 2 * i;
  *b = half ? i + r / 2 : 2 * i + 1;
}

// One row, one warp; any d and any even r.  pe == nullptr: a bad position.
template <typename T>
__device__ void norm_rope_row(const T* x, T* y, const T* gamma, const float* pe, int d, int r,
                              int half, float eps) {
  const int lane = threadIdx.x & 31;
  if (!pe) {
    for (int c = lane; c < d; c += 32) y[c] = static_cast<T>(0.f);
    return;
  }
  float ss = 0.f;
  for (int c = lane; c < d; c += 32) {
    const float v = static_cast<float>(x[c]);
    ss = fmaf(v, v, ss);
  }
  const float rstd = rsqrtf(warp_sum(ss) / d + eps);
  for (int i = lane; i < r / 2; i += 32) {
    int a, b;
    pair_columns(i, r, half, &a, &b);
    const float za = static_cast<float>(x[a]) * rstd * static_cast<float>(gamma[a]);
    const float zb = static_cast<float>(x[b]) * rstd * static_cast<float>(gamma[b]);
    const float sn = __ldg(pe + 2 * i), cs = __ldg(pe + 2 * i + 1);
    y[a] = static_cast<T>(za * cs - zb * sn);
    y[b] = static_cast<T>(zb * cs + za * sn);
  }
  for (int c = r + lane; c < d; c += 32)
    y[c] = static_cast<T>(static_cast<float>(x[c]) * rstd * static_cast<float>(gamma[c]));
}

struct TrainArgs {
  const void* x[2];        // Q, K
  int64_t ts[2];           // their token strides
  const void* gamma[2];
  const float* pe;
  int pe_rows, r, half;
  void* y[2];
  int B, L, heads[2], d, pos_offset;
  const int32_t* positions;
  float eps;
  unsigned* err;
  // backward
  const void* dy[2];
  int dy_f32[2];
  void* dx[2];
  int64_t dts[2];
  float* partial;  // [blocks][2][d]
};

// The table row of token `token` = b * L + l, or nullptr.
__device__ __forceinline__ const float* table_row(const TrainArgs& p, int64_t token, int l) {
  const int pos = p.positions ? __ldg(p.positions + token) : p.pos_offset + l;
  return pos >= 0 && pos < p.pe_rows ? p.pe + static_cast<int64_t>(pos) * p.r : nullptr;
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) norm_rope_any_kernel(const TrainArgs p) {
  const int per_token = p.heads[0] + p.heads[1];
  const int64_t rows = static_cast<int64_t>(p.B) * p.L * per_token;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); row < rows;
       row += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t token = row / per_token;
    const int hh = static_cast<int>(row - token * per_token);
    const int w = hh >= p.heads[0];
    const int h = w ? hh - p.heads[0] : hh;
    const int64_t b = token / p.L;
    const int l = static_cast<int>(token - b * p.L);
    const float* pe = table_row(p, token, l);
    if (!pe && (threadIdx.x & 31) == 0) atomicOr(p.err, kErrPosition);
    norm_rope_row(static_cast<const T*>(p.x[w]) + token * p.ts[w] + static_cast<int64_t>(h) * p.d,
                  static_cast<T*>(p.y[w]) + ((b * p.heads[w] + h) * p.L + l) * p.d,
                  static_cast<const T*>(p.gamma[w]), pe, p.d, p.r, p.half, p.eps);
  }
}

__device__ __forceinline__ float load_grad(const void* dy, int f32, int64_t i) {
  return f32 ? static_cast<const float*>(dy)[i]
             : __bfloat162float(static_cast<const __nv_bfloat16*>(dy)[i]);
}

// dx of every row, and per block the sums of dz * xh over its rows.
template <typename T>
__global__ void __launch_bounds__(32 * kWarps) norm_rope_any_bwd_kernel(const TrainArgs p) {
  __shared__ float sums[kWarps][kMaxD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pairs = p.r / 2;
  for (int w = 0; w < 2; ++w) {
    // this lane's columns: pairs lane, lane + 32, ... and tail columns
    float ga[4] = {}, gb[4] = {}, gt[8] = {};
    const T* gamma = static_cast<const T*>(p.gamma[w]);
    const int64_t rows = static_cast<int64_t>(p.B) * p.L * p.heads[w];
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp; row < rows;
         row += static_cast<int64_t>(gridDim.x) * kWarps) {
      const int64_t token = row / p.heads[w];
      const int h = static_cast<int>(row - token * p.heads[w]);
      const int64_t b = token / p.L;
      const int l = static_cast<int>(token - b * p.L);
      const T* x = static_cast<const T*>(p.x[w]) + token * p.ts[w] + static_cast<int64_t>(h) * p.d;
      T* dx = static_cast<T*>(p.dx[w]) + token * p.dts[w] + static_cast<int64_t>(h) * p.d;
      const int64_t dy0 = ((b * p.heads[w] + h) * p.L + l) * p.d;
      const float* pe = table_row(p, token, l);
      if (!pe) {
        if (lane == 0) atomicOr(p.err, kErrPosition);
        for (int c = lane; c < p.d; c += 32) dx[c] = static_cast<T>(0.f);
        continue;
      }
      float ss = 0.f;
      for (int c = lane; c < p.d; c += 32) {
        const float v = static_cast<float>(x[c]);
        ss = fmaf(v, v, ss);
      }
      const float rstd = rsqrtf(warp_sum(ss) / p.d + p.eps);
      float dot = 0.f;
      float xa[4], xb[4], ua[4], ub[4], xt[8], ut[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = lane + 32 * k;
        if (i >= pairs) continue;
        int a, c;
        pair_columns(i, p.r, p.half, &a, &c);
        const float sn = __ldg(pe + 2 * i), cs = __ldg(pe + 2 * i + 1);
        const float da = load_grad(p.dy[w], p.dy_f32[w], dy0 + a);
        const float db = load_grad(p.dy[w], p.dy_f32[w], dy0 + c);
        const float za = da * cs + db * sn, zb = db * cs - da * sn;
        xa[k] = static_cast<float>(x[a]) * rstd;
        xb[k] = static_cast<float>(x[c]) * rstd;
        ga[k] = fmaf(za, xa[k], ga[k]);
        gb[k] = fmaf(zb, xb[k], gb[k]);
        ua[k] = za * static_cast<float>(gamma[a]);
        ub[k] = zb * static_cast<float>(gamma[c]);
        dot = fmaf(ua[k], xa[k], fmaf(ub[k], xb[k], dot));
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = p.r + lane + 32 * k;
        if (c >= p.d) continue;
        const float z = load_grad(p.dy[w], p.dy_f32[w], dy0 + c);
        xt[k] = static_cast<float>(x[c]) * rstd;
        gt[k] = fmaf(z, xt[k], gt[k]);
        ut[k] = z * static_cast<float>(gamma[c]);
        dot = fmaf(ut[k], xt[k], dot);
      }
      const float m = warp_sum(dot) / p.d;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = lane + 32 * k;
        if (i >= pairs) continue;
        int a, c;
        pair_columns(i, p.r, p.half, &a, &c);
        dx[a] = static_cast<T>(rstd * (ua[k] - xa[k] * m));
        dx[c] = static_cast<T>(rstd * (ub[k] - xb[k] * m));
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = p.r + lane + 32 * k;
        if (c < p.d) dx[c] = static_cast<T>(rstd * (ut[k] - xt[k] * m));
      }
    }
    __syncthreads();  // the previous part's sums have been read
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = lane + 32 * k;
      if (i >= pairs) continue;
      int a, c;
      pair_columns(i, p.r, p.half, &a, &c);
      sums[warp][a] = ga[k];
      sums[warp][c] = gb[k];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = p.r + lane + 32 * k;
      if (c < p.d) sums[warp][c] = gt[k];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.d; c += 32 * kWarps) {
      float s = 0.f;
      for (int k = 0; k < kWarps; ++k) s += sums[k][c];
      p.partial[(static_cast<int64_t>(blockIdx.x) * 2 + w) * p.d + c] = s;
    }
  }
}

// dgamma[w][c] = sum over blocks of partial[block][w][c], in block order
// within a warp's share and then over the warps: fp64, one warp column set
// per block of 32 columns.
__global__ void __launch_bounds__(1024)
    dgamma_kernel(const float* __restrict__ partial, int blocks, int d, float* gq, float* gk) {
  __shared__ double sums[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;  // of 2 * d
  double s = 0.;
  if (col < 2 * d)
    for (int k = warp; k < blocks; k += 32) s += partial[static_cast<int64_t>(k) * 2 * d + col];
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < 2 * d) {
    double t = 0.;
    for (int k = 0; k < 32; ++k) t += sums[k][lane];
    float* out = col < d ? gq : gk;
    if (out) out[col < d ? col : col - d] = static_cast<float>(t);
  }
}

struct PagedArgs {
  const __nv_bfloat16 *q, *k, *v;
  int64_t qs, ks, vs;
  const __nv_bfloat16 *gq, *gk;
  const float* pe;
  int pe_rows, r, half;
  __nv_bfloat16* qo;
  PagesView pages;
  const int32_t* q_offsets;
  int T, H;
  float eps;
  unsigned* err;
};

__global__ void __launch_bounds__(32 * kWarps) norm_rope_paged_any_kernel(const PagedArgs p) {
  const int lane = threadIdx.x & 31;
  const PagesView& pg = p.pages;
  const int per_token = p.H + 2 * pg.kv_heads;
  const int64_t rows = static_cast<int64_t>(p.T) * per_token;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); row < rows;
       row += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int t = static_cast<int>(row / per_token);
    const int hh = static_cast<int>(row - static_cast<int64_t>(t) * per_token);
    const int b = sequence_of_token(p.q_offsets, pg.B, t);
    if (b >= pg.B) continue;
    const int q0 = __ldg(p.q_offsets + b), q1 = __ldg(p.q_offsets + b + 1);
    if (q0 < 0 || t < q0 || t >= q1 || q1 > p.T) {
      if (lane == 0) atomicOr(p.err, kErrPages);
      continue;
    }
    const int len = __ldg(pg.kv_len + b);
    const int n = q1 - q0;
    const int pos = len - n + (t - q0);
    int page = -1;
    if (len >= n && len <= (static_cast<int64_t>(pg.cols) << pg.page_shift))
      page = __ldg(pg.table + static_cast<int64_t>(b) * pg.cols + (pos >> pg.page_shift));
    const bool ok = page >= 0 && page < pg.num_pages && pos < p.pe_rows;
    if (!ok && lane == 0) atomicOr(p.err, pos < p.pe_rows ? kErrPages : kErrPosition);
    const float* pe = ok ? p.pe + static_cast<int64_t>(pos) * p.r : nullptr;
    const int d = pg.d;
    if (hh < p.H) {
      norm_rope_row(p.q + t * p.qs + static_cast<int64_t>(hh) * d,
                    p.qo + (static_cast<int64_t>(t) * p.H + hh) * d, p.gq, pe, d, p.r, p.half,
                    p.eps);
      continue;
    }
    if (!ok) continue;
    const int g = (hh - p.H) % pg.kv_heads;
    const int64_t at = page * pg.page_stride +
                       ((static_cast<int64_t>(g) << pg.page_shift) +
                        (pos & ((1 << pg.page_shift) - 1))) * d;
    if (hh < p.H + pg.kv_heads) {
      norm_rope_row(p.k + t * p.ks + static_cast<int64_t>(g) * d,
                    static_cast<__nv_bfloat16*>(pg.K) + at, p.gk, pe, d, p.r, p.half, p.eps);
    } else {
      const __nv_bfloat16* v = p.v + t * p.vs + static_cast<int64_t>(g) * d;
      for (int c = lane; c < d; c += 32) static_cast<__nv_bfloat16*>(pg.V)[at + c] = v[c];
    }
  }
}

int num_sms() {
  int dev = 0, v = 0;
  if (cudaGetDevice(&dev) == cudaSuccess &&
      cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && v > 0)
    return v;
  return 1;
}

unsigned grid_for(int64_t warps_wanted, int blocks_per_sm) {
  const int64_t want = (warps_wanted + kWarps - 1) / kWarps;
  const int64_t most = static_cast<int64_t>(blocks_per_sm) * num_sms();
  return static_cast<unsigned>(want < most ? want : most);
}

bool bad_ptr(const void* p, uintptr_t align) {
  return !p || (reinterpret_cast<uintptr_t>(p) & (align - 1));
}

// The checks that the three entry points share.  Resolves token strides.
mha_status check_rope(const float* pe, int pe_rows, int rope_dim, int pairing, int d, float eps,
                      int dtype) {
  if (dtype != MHA_BF16 && dtype != MHA_F32) return MHA_ERR_INVALID_ARG;
  if (pairing != MHA_ROPE_INTERLEAVED && pairing != MHA_ROPE_HALF) return MHA_ERR_INVALID_ARG;
  if (!(eps > 0.f) || isinf(eps)) return MHA_ERR_INVALID_ARG;
  if (d < 2 || rope_dim < 2 || rope_dim > d || rope_dim % 2 || pe_rows < 1)
    return MHA_ERR_INVALID_ARG;
  if (d > kMaxD) return MHA_ERR_UNSUPPORTED;
  return bad_ptr(pe, 8) ? MHA_ERR_INVALID_ARG : MHA_OK;
}

// Head rows that can be read as 16-byte vectors of whole pairs.
bool vector_rows(int d, int rope_dim) { return (d == 64 || d == 128) && rope_dim % 16 == 0; }

mha_status check_rows(const void* x, int64_t* ts, int heads, int d, int dtype, bool vec) {
  if (*ts == 0) *ts = static_cast<int64_t>(heads) * d;
  if (*ts < static_cast<int64_t>(heads) * d) return MHA_ERR_INVALID_ARG;
  if (bad_ptr(x, 16)) return MHA_ERR_INVALID_ARG;
  if (vec && (*ts * (dtype == MHA_BF16 ? 2 : 4)) % 16) return MHA_ERR_INVALID_ARG;
  return MHA_OK;
}

}  // namespace
}  // namespace mha

using namespace mha;

extern "C" {

mha_status qk_norm_rope_forward(const void* Q, int64_t q_token_stride, const void* K,
                                int64_t k_token_stride, const void* gamma_q, const void* gamma_k,
                                const float* pe, int pe_rows, int rope_dim, int pairing, void* Qo,
                                void* Ko, int B, int L, int H, int Hkv, int d, int pos_offset,
                                const int32_t* positions, float eps, mha_dtype dtype,
                                mha_stream stream) {
  if (B < 0 || L < 0 || H < 0 || Hkv < 0 || pos_offset < 0) return MHA_ERR_INVALID_ARG;
  mha_status st = check_rope(pe, pe_rows, rope_dim, pairing, d, eps, dtype);
  if (st != MHA_OK) return st;
  if (positions ? (reinterpret_cast<uintptr_t>(positions) & 3u) != 0
                : static_cast<int64_t>(pos_offset) + L > pe_rows)
    return MHA_ERR_INVALID_ARG;
  const bool vec = vector_rows(d, rope_dim);
  TrainArgs p{{Q, K}, {q_token_stride, k_token_stride}, {gamma_q, gamma_k}, pe, pe_rows, rope_dim,
              pairing, {Qo, Ko}, B, L, {H, Hkv}, d, pos_offset, positions, eps, nullptr};
  const bool empty = B == 0 || L == 0 || H + Hkv == 0;
  for (int w = 0; w < 2 && !empty; ++w) {
    if (p.heads[w] == 0) continue;
    st = check_rows(p.x[w], &p.ts[w], p.heads[w], d, dtype, vec);
    if (st != MHA_OK) return st;
    if (bad_ptr(p.gamma[w], 16) || bad_ptr(p.y[w], 16) || p.y[w] == p.x[w])
      return MHA_ERR_INVALID_ARG;
  }
  if (empty) return MHA_OK;
  DeviceCtl ctl;
  if (!device_ctl(&ctl)) return MHA_ERR_CUDA;
  p.err = ctl.err;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t rows = static_cast<int64_t>(B) * L * (H + Hkv);
  if (dtype == MHA_BF16)
    norm_rope_any_kernel<__nv_bfloat16><<<grid_for(rows, 16), 32 * kWarps, 0, s>>>(p);
  else
    norm_rope_any_kernel<float><<<grid_for(rows, 16), 32 * kWarps, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? MHA_OK : MHA_ERR_CUDA;
}

size_t qk_norm_rope_backward_workspace_bytes(int d) {
  if (d < 2 || d > kMaxD) return 0;
  return static_cast<size_t>(kMaxGradBlocks) * 2 * d * sizeof(float);
}

mha_status qk_norm_rope_backward(const void* Q, int64_t q_token_stride, const void* K,
                                 int64_t k_token_stride, const void* gamma_q, const void* gamma_k,
                                 const float* pe, int pe_rows, int rope_dim, int pairing,
                                 const void* dQo, const void* dKo, void* dQ,
                                 int64_t dq_token_stride, void* dK, int64_t dk_token_stride,
                                 float* dgamma_q, float* dgamma_k, int B, int L, int H, int Hkv,
                                 int d, int pos_offset, const int32_t* positions, float eps,
                                 mha_dtype dtype, mha_dtype dq_dtype, mha_dtype dk_dtype,
                                 void* workspace, size_t workspace_bytes, mha_stream stream) {
  if (B < 0 || L < 0 || H < 0 || Hkv < 0 || pos_offset < 0) return MHA_ERR_INVALID_ARG;
  mha_status st = check_rope(pe, pe_rows, rope_dim, pairing, d, eps, dtype);
  if (st != MHA_OK) return st;
  for (int t : {static_cast<int>(dq_dtype), static_cast<int>(dk_dtype)})
    if (t != MHA_BF16 && t != MHA_F32) return MHA_ERR_INVALID_ARG;
  if (positions ? (reinterpret_cast<uintptr_t>(positions) & 3u) != 0
                : static_cast<int64_t>(pos_offset) + L > pe_rows)
    return MHA_ERR_INVALID_ARG;
  const bool vec = vector_rows(d, rope_dim);
  TrainArgs p{{Q, K}, {q_token_stride, k_token_stride}, {gamma_q, gamma_k}, pe, pe_rows, rope_dim,
              pairing, {nullptr, nullptr}, B, L, {H, Hkv}, d, pos_offset, positions, eps, nullptr,
              {dQo, dKo}, {dq_dtype == MHA_F32, dk_dtype == MHA_F32}, {dQ, dK},
              {dq_token_stride, dk_token_stride}, static_cast<float*>(workspace)};
  float* dgamma[2] = {dgamma_q, dgamma_k};
  const bool rows_empty = B == 0 || L == 0;
  for (int w = 0; w < 2; ++w) {
    if (p.heads[w] == 0 && !dgamma[w]) continue;
    if (bad_ptr(dgamma[w], 16)) return MHA_ERR_INVALID_ARG;
    if (rows_empty || p.heads[w] == 0) continue;
    st = check_rows(p.x[w], &p.ts[w], p.heads[w], d, dtype, vec);
    if (st == MHA_OK) st = check_rows(p.dx[w], &p.dts[w], p.heads[w], d, dtype, vec);
    if (st != MHA_OK) return st;
    if (bad_ptr(p.gamma[w], 16) || bad_ptr(p.dy[w], 16) || p.dx[w] == p.x[w] || p.dx[w] == p.dy[w])
      return MHA_ERR_INVALID_ARG;
  }
  if (H + Hkv == 0) return MHA_OK;
  if (bad_ptr(workspace, 16) || workspace_bytes < qk_norm_rope_backward_workspace_bytes(d))
    return MHA_ERR_INVALID_ARG;
  DeviceCtl ctl;
  if (!device_ctl(&ctl)) return MHA_ERR_CUDA;
  p.err = ctl.err;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t rows = static_cast<int64_t>(B) * L * (H > Hkv ? H : Hkv);
  unsigned blocks = grid_for(rows, 4);
  if (blocks > kMaxGradBlocks) blocks = kMaxGradBlocks;
  if (blocks) {
    if (dtype == MHA_BF16)
      norm_rope_any_bwd_kernel<__nv_bfloat16><<<blocks, 32 * kWarps, 0, s>>>(p);
    else
      norm_rope_any_bwd_kernel<float><<<blocks, 32 * kWarps, 0, s>>>(p);
  }
  dgamma_kernel<<<(2 * d + 31) / 32, 1024, 0, s>>>(p.partial, static_cast<int>(blocks), d,
                                                   dgamma[0], dgamma[1]);
  return cudaGetLastError() == cudaSuccess ? MHA_OK : MHA_ERR_CUDA;
}

mha_status qk_norm_rope_paged(const void* Q, int64_t q_token_stride, const void* K,
                              int64_t k_token_stride, const void* V, int64_t v_token_stride,
                              const void* gamma_q, const void* gamma_k, const float* pe,
                              int pe_rows, int rope_dim, int pairing, void* Qo,
                              const mha_kv_pages* pages, int layer, const int32_t* q_offsets,
                              int T, int H, float eps, mha_stream stream) {
  mha_status st = validate_pages(pages);
  if (st != MHA_OK) return st;
  if (T < 0 || H < 1 || layer < 0 || layer >= pages->layers) return MHA_ERR_INVALID_ARG;
  if (pages->dtype != MHA_BF16) return MHA_ERR_UNSUPPORTED;
  const int d = pages->d, Hkv = pages->kv_heads;
  st = check_rope(pe, pe_rows, rope_dim, pairing, d, eps, MHA_BF16);
  if (st != MHA_OK) return st;
  if (!vector_rows(d, rope_dim)) return MHA_ERR_UNSUPPORTED;
  if (T == 0 || pages->B == 0) return MHA_OK;
  st = check_rows(Q, &q_token_stride, H, d, MHA_BF16, true);
  if (st == MHA_OK) st = check_rows(K, &k_token_stride, Hkv, d, MHA_BF16, true);
  if (st == MHA_OK) st = check_rows(V, &v_token_stride, Hkv, d, MHA_BF16, true);
  if (st != MHA_OK) return st;
  if (bad_ptr(gamma_q, 16) || bad_ptr(gamma_k, 16) || bad_ptr(Qo, 16) || Qo == Q ||
      bad_ptr(q_offsets, 4))
    return MHA_ERR_INVALID_ARG;
  DeviceCtl ctl;
  if (!device_ctl(&ctl)) return MHA_ERR_CUDA;
  auto bf = [](const void* q) { return static_cast<const __nv_bfloat16*>(q); };
  const PagedArgs p{bf(Q), bf(K), bf(V), q_token_stride, k_token_stride, v_token_stride,
                    bf(gamma_q), bf(gamma_k), pe, pe_rows, rope_dim, pairing,
                    static_cast<__nv_bfloat16*>(Qo), pages_view(*pages, layer), q_offsets, T, H,
                    eps, ctl.err};
  const int64_t rows = static_cast<int64_t>(T) * (H + 2 * Hkv);
  norm_rope_paged_any_kernel<<<grid_for(rows, 16), 32 * kWarps, 0,
                               reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? MHA_OK : MHA_ERR_CUDA;
}

}  // extern "C"
