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
//
// Head sizes 64 and 128 (with rope_dim a multiple of 16) take the vector
// kernels: a row's 16-byte vectors lie two to a lane, in 4 or 8 lanes, so a
// warp has 8 or 4 rows in flight; a lane's two vectors are the two halves of
// its column pairs when the pairing is half-wise, so the rotation needs no
// exchange, and the sums of a row take 2 or 3 shuffles.  Other sizes take the
// element-wise kernels, one warp per row.
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

// ------------------------------------------------------------- vector kernels

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(h[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint4 u;
  u.x = pack_bf16x2(v[0], v[1]);
  u.y = pack_bf16x2(v[2], v[3]);
  u.z = pack_bf16x2(v[4], v[5]);
  u.w = pack_bf16x2(v[6], v[7]);
  *reinterpret_cast<uint4*>(p) = u;
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// A lane's place in a row of D columns: vectors `a` and `b` (in elements).
template <int D>
struct VecLane {
  static constexpr int kLanes = D / 16;        // lanes per row
  static constexpr int kRows = 32 / kLanes;    // rows per warp
  int a, b;
  bool turns;  // its columns are rotated

  __device__ __forceinline__ explicit VecLane(int r) {
    const int j = (threadIdx.x & 31) % kLanes;
    turns = j < r / 16;
    // rotated: a column pair's halves; the rest: two neighbours
    a = turns ? 8 * j : r + 16 * (j - r / 16);
    b = turns ? 8 * j + r / 2 : a + 8;
  }
};

// Sines and cosines of a lane's eight pairs: half-wise pairs (a + i, b + i),
// or interleaved ones, four in each vector.
struct Turns {
  float sn[8], cs[8];

  __device__ __forceinline__ void load(const float* pe, int a, int b, bool turns, int half) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float4 v = make_float4(0.f, 1.f, 0.f, 1.f);
      // pairs a .. a+7 of the table, or those at columns a .. and b ..
      if (turns)
        v = __ldg(reinterpret_cast<const float4*>(half ? pe + 2 * a : k < 2 ? pe + a : pe + b - 8) +
                  k);
      sn[2 * k] = v.x, cs[2 * k] = v.y, sn[2 * k + 1] = v.z, cs[2 * k + 1] = v.w;
    }
  }

  // Rotate by the angle (sign 1) or its opposite (sign -1).
  __device__ __forceinline__ void turn(float (&x)[8], float (&y)[8], int half, float sign) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float& p = half ? x[k] : k < 4 ? x[2 * k] : y[2 * (k - 4)];
      float& q = half ? y[k] : k < 4 ? x[2 * k + 1] : y[2 * (k - 4) + 1];
      const float s = sign * sn[k], u = p, v = q;
      p = u * cs[k] - v * s;
      q = v * cs[k] + u * s;
    }
  }
};

template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int s = D / 32; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// One row per group of lanes.  Every lane of the warp takes part; `live`
// lanes hold x, the others zeros.
template <int D, typename T>
__device__ __forceinline__ void norm_rope_vec(float (&x)[8], float (&y)[8], const T* gamma,
                                              const VecLane<D>& at, const Turns& turns, int half,
                                              float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
  const float rstd = rsqrtf(row_sum<D>(ss) * (1.f / D) + eps);
  float ga[8], gb[8];
  load8(gamma + at.a, ga);
  load8(gamma + at.b, gb);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] *= rstd * ga[i];
    y[i] *= rstd * gb[i];
  }
  turns.turn(x, y, half, 1.f);
}

// Rows of one tensor, of `heads` heads a token.
struct RowPlace {
  uint32_t token, h, b, l;
  __device__ __forceinline__ RowPlace(uint32_t row, uint32_t heads, uint32_t L) {
    token = row / heads;
    h = row - token * heads;
    b = token / L;
    l = token - b * L;
  }
};

template <int D, typename T, int HALF>
__global__ void __launch_bounds__(32 * kWarps) norm_rope_vec_kernel(const TrainArgs p) {
  using V = VecLane<D>;
  const V at(p.r);
  const int lane = threadIdx.x & 31;
  const uint32_t tokens = static_cast<uint32_t>(p.B) * p.L;
  const uint32_t rows[2] = {tokens * p.heads[0], tokens * p.heads[1]};
  const uint32_t items0 = (rows[0] + V::kRows - 1) / V::kRows;
  const uint32_t items = items0 + (rows[1] + V::kRows - 1) / V::kRows;
  for (uint32_t it = blockIdx.x * kWarps + (threadIdx.x >> 5); it < items;
       it += gridDim.x * kWarps) {
    const int w = it >= items0;  // queries, then keys: uniform in a warp
    const uint32_t row = (w ? it - items0 : it) * V::kRows + lane / V::kLanes;
    const bool live = row < rows[w];
    const RowPlace at_row(live ? row : 0, p.heads[w], p.L);
    const T* x = static_cast<const T*>(p.x[w]) + at_row.token * p.ts[w] +
                 static_cast<int64_t>(at_row.h) * D;
    float a[8] = {}, b[8] = {};
    if (live) {
      load8(x + at.a, a);
      load8(x + at.b, b);
    }
    const float* pe = table_row(p, at_row.token, at_row.l);
    if (live && !pe) atomicOr(p.err, kErrPosition);
    Turns turns;
    turns.load(pe, at.a, at.b, at.turns && pe, HALF);
    norm_rope_vec<D>(a, b, static_cast<const T*>(p.gamma[w]), at, turns, HALF, p.eps);
    if (live) {
      T* y = static_cast<T*>(p.y[w]) +
             ((static_cast<int64_t>(at_row.b) * p.heads[w] + at_row.h) * p.L + at_row.l) * D;
      if (!pe) {
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = b[i] = 0.f;
      }
      store8(y + at.a, a);
      store8(y + at.b, b);
    }
  }
}

// dx of every row; per block the sums of dz * xh over its rows, first over a
// lane's rows, then over the row groups of a warp, then over the warps: a
// fixed order.
template <int D, typename T, int HALF>
__global__ void __launch_bounds__(32 * kWarps) norm_rope_vec_bwd_kernel(const TrainArgs p) {
  using V = VecLane<D>;
  __shared__ float sums[kWarps][D];
  const V at(p.r);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t tokens = static_cast<uint32_t>(p.B) * p.L;
  for (int w = 0; w < 2; ++w) {
    float g0[8] = {}, g1[8] = {}, ga[8], gb[8];
    const uint32_t rows = tokens * p.heads[w];
    const uint32_t items = (rows + V::kRows - 1) / V::kRows;
    if (rows) {
      load8(static_cast<const T*>(p.gamma[w]) + at.a, ga);
      load8(static_cast<const T*>(p.gamma[w]) + at.b, gb);
    }
    for (uint32_t it = blockIdx.x * kWarps + warp; it < items; it += gridDim.x * kWarps) {
      const uint32_t row = it * V::kRows + lane / V::kLanes;
      const RowPlace at_row(row < rows ? row : 0, p.heads[w], p.L);
      const float* pe = table_row(p, at_row.token, at_row.l);
      if (row < rows && !pe) atomicOr(p.err, kErrPosition);
      const bool live = row < rows && pe;
      const int64_t in = static_cast<int64_t>(at_row.h) * D;
      const int64_t dy0 =
          ((static_cast<int64_t>(at_row.b) * p.heads[w] + at_row.h) * p.L + at_row.l) * D;
      float a[8] = {}, b[8] = {}, u[8] = {}, v[8] = {};
      if (live) {
        const T* x = static_cast<const T*>(p.x[w]) + at_row.token * p.ts[w] + in;
        load8(x + at.a, a);
        load8(x + at.b, b);
        if (p.dy_f32[w]) {
          load8(static_cast<const float*>(p.dy[w]) + dy0 + at.a, u);
          load8(static_cast<const float*>(p.dy[w]) + dy0 + at.b, v);
        } else {
          load8(static_cast<const __nv_bfloat16*>(p.dy[w]) + dy0 + at.a, u);
          load8(static_cast<const __nv_bfloat16*>(p.dy[w]) + dy0 + at.b, v);
        }
      }
      Turns turns;
      turns.load(pe, at.a, at.b, at.turns && pe, HALF);
      turns.turn(u, v, HALF, -1.f);
      float ss = 0.f, ux = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
        ux = fmaf(u[i] * ga[i], a[i], fmaf(v[i] * gb[i], b[i], ux));
      }
      ss = row_sum<D>(ss);
      ux = row_sum<D>(ux);
      const float rstd = rsqrtf(ss * (1.f / D) + p.eps);
      const float m = rstd * rstd * ux * (1.f / D);  // mean(u * xh) * rstd
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g0[i] = fmaf(u[i], a[i] * rstd, g0[i]);
        g1[i] = fmaf(v[i], b[i] * rstd, g1[i]);
        a[i] = rstd * (u[i] * ga[i] - a[i] * m);
        b[i] = rstd * (v[i] * gb[i] - b[i] * m);
      }
      if (row < rows) {
        T* dx = static_cast<T*>(p.dx[w]) + at_row.token * p.dts[w] + in;
        store8(dx + at.a, a);
        store8(dx + at.b, b);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int s = V::kLanes; s < 32; s <<= 1) {
        g0[i] += __shfl_xor_sync(0xffffffffu, g0[i], s);
        g1[i] += __shfl_xor_sync(0xffffffffu, g1[i], s);
      }
    }
    __syncthreads();  // the previous part's sums have been read
    if (lane < V::kLanes) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sums[warp][at.a + i] = g0[i];
        sums[warp][at.b + i] = g1[i];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += 32 * kWarps) {
      float s = 0.f;
      for (int k = 0; k < kWarps; ++k) s += sums[k][c];
      p.partial[(static_cast<int64_t>(blockIdx.x) * 2 + w) * D + c] = s;
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

constexpr int kMaxBlockTokens = 8;  // one warp looks one token up

// A block takes block_tokens tokens: their sequences, positions and page rows
// are looked up once, a warp per token, then all warps take their rows,
// queries, keys and values, kRows at a time.
template <int D, int HALF>
__global__ void __launch_bounds__(32 * kWarps)
    norm_rope_paged_kernel(const PagedArgs p, int block_tokens) {
  using V = VecLane<D>;
  __shared__ int64_t row_at[kMaxBlockTokens];  // the token's pool row of head 0, in elements
  __shared__ int pos_of[kMaxBlockTokens];      // -1: no sequence's, -2: a bad entry
  const PagesView& pg = p.pages;
  const V at(p.r);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = blockIdx.x * block_tokens;
  const int tokens = min(block_tokens, p.T - t0);
  if (warp < tokens) {
    const int t = t0 + warp;
    const int b = sequence_of_token(p.q_offsets, pg.B, t);
    int pos = -1;
    int64_t row = 0;
    if (b < pg.B) {
      const int q0 = __ldg(p.q_offsets + b), q1 = __ldg(p.q_offsets + b + 1);
      const int len = __ldg(pg.kv_len + b);
      if (q0 < 0 || t < q0 || t >= q1 || q1 > p.T) {
        if (lane == 0) atomicOr(p.err, kErrPages);
      } else {
        const int n = q1 - q0;
        int page = -1;
        pos = len - n + (t - q0);
        if (len >= n && len <= (static_cast<int64_t>(pg.cols) << pg.page_shift))
          page = __ldg(pg.table + static_cast<int64_t>(b) * pg.cols + (pos >> pg.page_shift));
        if (page < 0 || page >= pg.num_pages || pos >= p.pe_rows) {
          if (lane == 0) atomicOr(p.err, kErrPages);
          pos = -2;
        } else {
          row = page * pg.page_stride + static_cast<int64_t>(pos & ((1 << pg.page_shift) - 1)) * D;
        }
      }
    }
    if (lane == 0) {
      row_at[warp] = row;
      pos_of[warp] = pos;
    }
  }
  __syncthreads();
  const int head_rows = D << pg.page_shift;  // elements from kv head to kv head of a page
  const int heads[3] = {p.H, pg.kv_heads, pg.kv_heads};
#pragma unroll
  for (int w = 0; w < 3; ++w) {  // queries, keys, values
    const int rows = tokens * heads[w];
    for (int r0 = warp * V::kRows; r0 < rows; r0 += kWarps * V::kRows) {
      const int row = r0 + lane / V::kLanes;
      const int k = row < rows ? row / heads[w] : 0;
      const int h = row - k * heads[w];
      const int pos = row < rows ? pos_of[k] : -1;
      const int64_t t = t0 + k;
      const __nv_bfloat16* x = (w == 0 ? p.q + t * p.qs : w == 1 ? p.k + t * p.ks : p.v + t * p.vs) +
                               static_cast<int64_t>(h) * D;
      const int64_t out = w == 0 ? (t * p.H + h) * D
                                 : row_at[k] + static_cast<int64_t>(h) * head_rows;
      if (w == 2) {
        if (pos < 0) continue;
        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(pg.V) + out;
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(x + at.a));
        const uint4 b = __ldg(reinterpret_cast<const uint4*>(x + at.b));
        *reinterpret_cast<uint4*>(y + at.a) = a;
        *reinterpret_cast<uint4*>(y + at.b) = b;
        continue;
      }
      float a[8] = {}, b[8] = {};
      if (pos >= 0) {
        load8(x + at.a, a);
        load8(x + at.b, b);
      }
      Turns turns;
      turns.load(p.pe + static_cast<int64_t>(max(pos, 0)) * p.r, at.a, at.b, at.turns && pos >= 0,
                 HALF);
      norm_rope_vec<D>(a, b, w == 0 ? p.gq : p.gk, at, turns, HALF, p.eps);
      // a bad entry: the query row is zeros (a and b are), the page untouched
      if (pos == -1 || (w == 1 && pos < 0)) continue;
      __nv_bfloat16* y = w == 0 ? p.qo + out : static_cast<__nv_bfloat16*>(pg.K) + out;
      store8(y + at.a, a);
      store8(y + at.b, b);
    }
    __syncwarp();
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
  return bad_ptr(pe, 16) ? MHA_ERR_INVALID_ARG : MHA_OK;
}

// Head rows that can be read as 16-byte vectors of whole pairs.
bool vector_rows(int d, int rope_dim) { return (d == 64 || d == 128) && rope_dim % 16 == 0; }

int64_t vec_items(int64_t rows, int d) { return (rows + 512 / d - 1) / (512 / d); }

struct ForwardKernels {
  template <int D, typename T, int HALF>
  static constexpr auto get() { return norm_rope_vec_kernel<D, T, HALF>; }
};
struct BackwardKernels {
  template <int D, typename T, int HALF>
  static constexpr auto get() { return norm_rope_vec_bwd_kernel<D, T, HALF>; }
};

template <typename K, typename T>
void (*vec_kernel_of(int d, int half))(const TrainArgs) {
  if (d == 64) return half ? K::template get<64, T, 1>() : K::template get<64, T, 0>();
  return half ? K::template get<128, T, 1>() : K::template get<128, T, 0>();
}

template <typename K>
void (*vec_kernel(int d, int dtype, int half))(const TrainArgs) {
  return dtype == MHA_BF16 ? vec_kernel_of<K, __nv_bfloat16>(d, half)
                           : vec_kernel_of<K, float>(d, half);
}

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
  if (static_cast<int64_t>(B) * L * (H + static_cast<int64_t>(Hkv)) > 0x7fffffffLL)
    return MHA_ERR_UNSUPPORTED;
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
  if (vec) {
    const auto kern = vec_kernel<ForwardKernels>(d, dtype, pairing);
    kern<<<grid_for(vec_items(rows, d), 8), 32 * kWarps, 0, s>>>(p);
  } else if (dtype == MHA_BF16) {
    norm_rope_any_kernel<__nv_bfloat16><<<grid_for(rows, 16), 32 * kWarps, 0, s>>>(p);
  } else {
    norm_rope_any_kernel<float><<<grid_for(rows, 16), 32 * kWarps, 0, s>>>(p);
  }
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
  if (static_cast<int64_t>(B) * L * (H + static_cast<int64_t>(Hkv)) > 0x7fffffffLL)
    return MHA_ERR_UNSUPPORTED;
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
  unsigned blocks = grid_for(vec ? vec_items(rows, d) : rows, 4);
  if (blocks > kMaxGradBlocks) blocks = kMaxGradBlocks;
  if (blocks) {
    if (vec)
      vec_kernel<BackwardKernels>(d, dtype, pairing)<<<blocks, 32 * kWarps, 0, s>>>(p);
    else if (dtype == MHA_BF16)
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
  // a block per token until the SMs have four each, then up to eight tokens
  const int64_t per_block = T / (4 * static_cast<int64_t>(num_sms()));
  const int block_tokens = per_block < 1 ? 1 : per_block < kMaxBlockTokens
                                                   ? static_cast<int>(per_block)
                                                   : kMaxBlockTokens;
  const unsigned grid = static_cast<unsigned>((T + block_tokens - 1) / block_tokens);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d == 64 && pairing == MHA_ROPE_HALF)
    norm_rope_paged_kernel<64, 1><<<grid, 32 * kWarps, 0, s>>>(p, block_tokens);
  else if (d == 64)
    norm_rope_paged_kernel<64, 0><<<grid, 32 * kWarps, 0, s>>>(p, block_tokens);
  else if (pairing == MHA_ROPE_HALF)
    norm_rope_paged_kernel<128, 1><<<grid, 32 * kWarps, 0, s>>>(p, block_tokens);
  else
    norm_rope_paged_kernel<128, 0><<<grid, 32 * kWarps, 0, s>>>(p, block_tokens);
  return cudaGetLastError() == cudaSuccess ? MHA_OK : MHA_ERR_CUDA;
}

}  // extern "C"
