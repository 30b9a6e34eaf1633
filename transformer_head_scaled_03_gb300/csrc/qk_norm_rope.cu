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
// About ten flops per element moved: HBM sets the floor, or the launch when
// there are few rows.  What bounds the kernels is latency, by the counters:
// DRAM at 45 (append) to 66 % of its nominal rate, 25 to 41 % of the warps
// resident, half of the issue slots in use.
//
// Head sizes 64 and 128 (with rope_dim a multiple of 16) take the vector
// kernels: a row's 16-byte vectors lie two to a lane, in 4 or 8 lanes, so a
// warp has 8 or 4 rows in flight; a lane's two vectors are the two halves of
// its column pairs when the pairing is half-wise, so the rotation needs no
// exchange, and the sums of a row take 2 or 3 shuffles.  Other sizes take the
// element-wise kernels, one warp per row.
//
// Measured with nothing in L2, bytes of the operator by time, B16 L2048
// H16 + 16 d64 bf16: forward 51 us (5.2 TB/s; 33 % occupancy at 77 registers),
// gradient with dQ in fp32 106 us (4.4 TB/s; 25 % at 128 registers, and two
// phases, queries and keys); fp32 109 and 172 us (5.0 and 4.7 TB/s).
// B4 L4096 H32 + 8 d128: 66 and 122 us, fp32 135 and 207.  The element-wise
// kernels at the first shape with d = 96: 463 and 1,242 us, 8 to 12 times the
// bytes' time: two bytes a lane, and x read twice; with d = 256 616 and 1,584
// us, 4 to 6 times.  Appending 8,262 tokens of 32 + 8 + 8 heads: 48 us (203 MB,
// 4.2 TB/s: a row is loaded, computed and stored before the next is requested);
// four tokens: 3 us.
#include <math.h>
#include <stdint.h>

#include <cuda_bf16.h>

#include "internal.h"
#include "kv_pages.cuh"
#include "ptx_pdl.cuh"

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
  pdl_launch_dependents();
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

__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}

// Eight elements as loaded (requested early) and as four fp32 pairs.
template <typename T>
struct Raw8;

template <>
struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void zero() { u = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    u = __ldg(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void get(float2 (&v)[4]) const {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __bfloat1622float2(h[i]);
  }
};

template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float2 (&v)[4]) const {
    v[0] = make_float2(a.x, a.y), v[1] = make_float2(a.z, a.w);
    v[2] = make_float2(b.x, b.y), v[3] = make_float2(b.z, b.w);
  }
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, float2 (&v)[4]) {
  Raw8<T> r;
  r.load(p);
  r.get(v);
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float2 (&v)[4]) {
  uint4 u;
  u.x = pack_bf16x2(v[0].x, v[0].y);
  u.y = pack_bf16x2(v[1].x, v[1].y);
  u.z = pack_bf16x2(v[2].x, v[2].y);
  u.w = pack_bf16x2(v[3].x, v[3].y);
  *reinterpret_cast<uint4*>(p) = u;
}

__device__ __forceinline__ void store8(float* p, const float2 (&v)[4]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
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
  float2 sn[4], cs[4];

  __device__ __forceinline__ void load(const float* pe, int a, int b, bool turns, int half) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float4 v = make_float4(0.f, 1.f, 0.f, 1.f);
      // pairs a .. a+7 of the table, or those at columns a .. and b ..
      if (turns)
        v = __ldg(reinterpret_cast<const float4*>(half ? pe + 2 * a : k < 2 ? pe + a : pe + b - 8) +
                  k);
      sn[k] = make_float2(v.x, v.z);
      cs[k] = make_float2(v.y, v.w);
    }
  }

  // Rotate by the angle, or by its opposite.
  template <int HALF, bool BACK>
  __device__ __forceinline__ void turn(float2 (&x)[4], float2 (&y)[4]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (HALF) {
        const float2 s = BACK ? make_float2(-sn[k].x, -sn[k].y) : sn[k];
        const float2 u = x[k], v = y[k];
        x[k] = ffma2(v, make_float2(-s.x, -s.y), fmul2(u, cs[k]));
        y[k] = ffma2(u, s, fmul2(v, cs[k]));
      } else {
        // pairs 2k and 2k + 1: those of x, then those of y
        float2& p = k < 2 ? x[2 * k] : y[2 * k - 4];
        float2& q = k < 2 ? x[2 * k + 1] : y[2 * k - 3];
        const float s0 = BACK ? -sn[k].x : sn[k].x, s1 = BACK ? -sn[k].y : sn[k].y;
        p = make_float2(fmaf(p.x, cs[k].x, -p.y * s0), fmaf(p.y, cs[k].x, p.x * s0));
        q = make_float2(fmaf(q.x, cs[k].y, -q.y * s1), fmaf(q.y, cs[k].y, q.x * s1));
      }
    }
  }
};

template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int s = D / 32; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// The sum of a lane's products.
__device__ __forceinline__ float dot8(const float2 (&a)[4], const float2 (&b)[4]) {
  float2 s = fmul2(a[0], b[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = ffma2(a[i], b[i], s);
  return s.x + s.y;
}

__device__ __forceinline__ void scale8(float2 (&a)[4], const float2 (&g)[4], float s) {
  const float2 s2 = make_float2(s, s);
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = fmul2(fmul2(a[i], s2), g[i]);
}

// One row per group of lanes.  Every lane of the warp takes part, those
// without a row on zeros.
template <int D, int HALF, typename T>
__device__ __forceinline__ void norm_rope_vec(float2 (&x)[4], float2 (&y)[4], const T* gamma,
                                              const VecLane<D>& at, const Turns& turns,
                                              float eps) {
  const float ss = row_sum<D>(dot8(x, x) + dot8(y, y));
  const float rstd = rsqrtf(ss * (1.f / D) + eps);
  float2 ga[4], gb[4];
  load8(gamma + at.a, ga);
  load8(gamma + at.b, gb);
  scale8(x, ga, rstd);
  scale8(y, gb, rstd);
  turns.turn<HALF, false>(x, y);
}

// How a warp's row groups take the heads of tokens: as many whole tokens at a
// time as fit, or one token over several rounds.  A row group keeps its token,
// so its sines and cosines are loaded once for all of the token's heads.
struct Rounds {
  int tokens;  // tokens a warp takes at a time
  int cols;    // row groups to a token
  int rounds;  // rounds of heads to a token
  __device__ __forceinline__ Rounds(int heads, int groups) {
    tokens = heads < groups ? groups / heads : 1;
    cols = heads < groups ? heads : groups;
    rounds = (heads + groups - 1) / groups;
  }
};

// A row group's walk over its tokens and, within a token, its rounds.
// `parts` warps share a token's rounds (when there are few tokens).
struct Walk {
  uint32_t it, token, b, l;
  int round;
  bool here;        // the row group has a token
  const float* pe;  // its table row, nullptr without one

  __device__ __forceinline__ void enter(const TrainArgs& p, const Rounds& rd, int gt, int parts,
                                        uint32_t tokens, uint32_t items) {
    const uint32_t tg = it / parts;
    round = static_cast<int>(it - tg * parts);
    token = tg * rd.tokens + gt;
    here = it < items && gt < rd.tokens && token < tokens;
    if (!here) token = 0;
    b = token / p.L;
    l = token - b * p.L;
    pe = here ? table_row(p, token, l) : nullptr;
  }
  // On to the next round; true when that is another token's.
  __device__ __forceinline__ bool next(const TrainArgs& p, const Rounds& rd, int gt, int parts,
                                       uint32_t tokens, uint32_t items) {
    round += parts;
    if (round < rd.rounds) return false;
    it += gridDim.x * kWarps;
    enter(p, rd, gt, parts, tokens, items);
    return true;
  }
};

template <int D, typename T, int HALF>
__global__ void __launch_bounds__(32 * kWarps)
    norm_rope_vec_kernel(const TrainArgs p, int parts) {
  using V = VecLane<D>;
  const V at(p.r);
  const int group = (threadIdx.x & 31) / V::kLanes;
  const int heads = p.heads[0] + p.heads[1];
  const Rounds rd(heads, V::kRows);
  const uint32_t tokens = static_cast<uint32_t>(p.B) * p.L;
  const uint32_t items = (tokens + rd.tokens - 1) / rd.tokens * parts;
  const int gt = group / rd.cols, h0 = group - gt * rd.cols;
  Walk c;
  c.it = blockIdx.x * kWarps + (threadIdx.x >> 5);
  c.enter(p, rd, gt, parts, tokens, items);
  auto request = [&](const Walk& k, Raw8<T>& ra, Raw8<T>& rb) {
    const int h = h0 + k.round * V::kRows;
    ra.zero();
    rb.zero();
    if (!k.here || h >= heads) return;
    const int w = h >= p.heads[0];
    const T* x = static_cast<const T*>(p.x[w]) + k.token * p.ts[w] +
                 static_cast<int64_t>(w ? h - p.heads[0] : h) * D;
    ra.load(x + at.a);
    rb.load(x + at.b);
  };
  Raw8<T> ra, rb;
  request(c, ra, rb);
  Turns turns;
  turns.load(c.pe, at.a, at.b, at.turns && c.pe, HALF);
  while (c.it < items) {
    float2 x[4], y[4];
    ra.get(x);
    rb.get(y);
    Walk n = c;
    const bool other = n.next(p, rd, gt, parts, tokens, items);
    request(n, ra, rb);  // the next rows, while these are computed
    const int h = h0 + c.round * V::kRows;
    const int w = h >= p.heads[0];
    const int hw = w ? h - p.heads[0] : h;
    const bool live = c.here && h < heads;
    norm_rope_vec<D, HALF>(
        x, y, static_cast<const T*>(live ? p.gamma[w] : p.gamma[h0 >= p.heads[0]]), at, turns,
        p.eps);
    if (live) {
      T* out = static_cast<T*>(p.y[w]) +
               ((static_cast<int64_t>(c.b) * p.heads[w] + hw) * p.L + c.l) * D;
      if (!c.pe) {
        atomicOr(p.err, kErrPosition);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = y[i] = make_float2(0.f, 0.f);
      }
      store8(out + at.a, x);
      store8(out + at.b, y);
    }
    c = n;
    if (other) turns.load(c.pe, at.a, at.b, at.turns && c.pe, HALF);
  }
}

// dx of every row; per block the sums of dz * xh over its rows, first over a
// lane's rows, then over the row groups of a warp, then over the warps: a
// fixed order.
template <int D, typename T, typename TG, int HALF>
__device__ __forceinline__ void norm_rope_vec_bwd_part(const TrainArgs& p, int w, int parts,
                                                       float2 (&g0)[4], float2 (&g1)[4]) {
  using V = VecLane<D>;
  const V at(p.r);
  const int group = (threadIdx.x & 31) / V::kLanes;
  const int heads = p.heads[w];
  const Rounds rd(heads, V::kRows);
  const uint32_t tokens = static_cast<uint32_t>(p.B) * p.L;
  const uint32_t items = (tokens + rd.tokens - 1) / rd.tokens * parts;
  const int gt = group / rd.cols, h0 = group - gt * rd.cols;
  Walk c;
  c.it = blockIdx.x * kWarps + (threadIdx.x >> 5);
  c.enter(p, rd, gt, parts, tokens, items);
  auto request = [&](const Walk& k, Raw8<T>& ra, Raw8<T>& rb, Raw8<TG>& ru, Raw8<TG>& rv) {
    const int h = h0 + k.round * V::kRows;
    ra.zero();
    rb.zero();
    ru.zero();
    rv.zero();
    if (!k.pe || h >= heads) return;
    const T* x = static_cast<const T*>(p.x[w]) + k.token * p.ts[w] + static_cast<int64_t>(h) * D;
    const TG* dy = static_cast<const TG*>(p.dy[w]) +
                   ((static_cast<int64_t>(k.b) * heads + h) * p.L + k.l) * D;
    ra.load(x + at.a);
    rb.load(x + at.b);
    ru.load(dy + at.a);
    rv.load(dy + at.b);
  };
  Raw8<T> ra, rb;
  Raw8<TG> ru, rv;
  request(c, ra, rb, ru, rv);
  Turns turns;
  turns.load(c.pe, at.a, at.b, at.turns && c.pe, HALF);
  while (c.it < items) {
    float2 x[4], y[4], u[4], v[4];
    ra.get(x);
    rb.get(y);
    ru.get(u);
    rv.get(v);
    Walk n = c;
    const bool other = n.next(p, rd, gt, parts, tokens, items);
    request(n, ra, rb, ru, rv);  // the next rows, while these are computed
    turns.turn<HALF, true>(u, v);
    const float ss = row_sum<D>(dot8(x, x) + dot8(y, y));
    const float rstd = rsqrtf(ss * (1.f / D) + p.eps);
    const float2 rstd2 = make_float2(rstd, rstd);
    float2 ga[4], gb[4];
    load8(static_cast<const T*>(p.gamma[w]) + at.a, ga);
    load8(static_cast<const T*>(p.gamma[w]) + at.b, gb);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = fmul2(x[i], rstd2);
      y[i] = fmul2(y[i], rstd2);
      g0[i] = ffma2(u[i], x[i], g0[i]);
      g1[i] = ffma2(v[i], y[i], g1[i]);
      u[i] = fmul2(u[i], ga[i]);
      v[i] = fmul2(v[i], gb[i]);
    }
    const float m = row_sum<D>(dot8(u, x) + dot8(v, y)) * (-1.f / D);
    const float2 m2 = make_float2(m, m);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = fmul2(rstd2, ffma2(x[i], m2, u[i]));
      y[i] = fmul2(rstd2, ffma2(y[i], m2, v[i]));
    }
    const int h = h0 + c.round * V::kRows;
    if (c.here && h < heads) {
      if (!c.pe) {
        // zeros so far, unless gamma is not finite
        atomicOr(p.err, kErrPosition);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = y[i] = make_float2(0.f, 0.f);
      }
      T* dx = static_cast<T*>(p.dx[w]) + c.token * p.dts[w] + static_cast<int64_t>(h) * D;
      store8(dx + at.a, x);
      store8(dx + at.b, y);
    }
    c = n;
    if (other) turns.load(c.pe, at.a, at.b, at.turns && c.pe, HALF);
  }
}

template <int D, typename T, int HALF>
__global__ void __launch_bounds__(32 * kWarps)
    norm_rope_vec_bwd_kernel(const TrainArgs p, int parts) {
  using V = VecLane<D>;
  __shared__ float2 sums[kWarps][D / 2];
  pdl_launch_dependents();
  const V at(p.r);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int w = 0; w < 2; ++w) {
    float2 g0[4] = {}, g1[4] = {};
    if (p.heads[w] && p.dy_f32[w])
      norm_rope_vec_bwd_part<D, T, float, HALF>(p, w, parts, g0, g1);
    else if (p.heads[w])
      norm_rope_vec_bwd_part<D, T, __nv_bfloat16, HALF>(p, w, parts, g0, g1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int s = V::kLanes; s < 32; s <<= 1) {
        g0[i].x += __shfl_xor_sync(0xffffffffu, g0[i].x, s);
        g0[i].y += __shfl_xor_sync(0xffffffffu, g0[i].y, s);
        g1[i].x += __shfl_xor_sync(0xffffffffu, g1[i].x, s);
        g1[i].y += __shfl_xor_sync(0xffffffffu, g1[i].y, s);
      }
    }
    __syncthreads();  // the previous part's sums have been read
    if (lane < V::kLanes) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sums[warp][at.a / 2 + i] = g0[i];
        sums[warp][at.b / 2 + i] = g1[i];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += 32 * kWarps) {
      float s = 0.f;
      for (int k = 0; k < kWarps; ++k) s += reinterpret_cast<const float*>(sums[k])[c];
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
  pdl_wait();
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

// A block takes block_tokens tokens (gridDim.y blocks share them when there
// are few): their sequences, positions and page rows are looked up once, a
// warp per token, then all warps take their rows, queries, keys and values,
// kRows at a time.
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
      // ascending offsets put t into [q0, q1), or ahead of the first sequence,
      // where it is nobody's
      if (q0 < 0 || q1 < q0 || q1 > p.T || t >= q1 || (b > 0 && t < q0)) {
        if (lane == 0) atomicOr(p.err, kErrPages);
      } else if (t >= q0) {
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
  const int q_items = (tokens * p.H + V::kRows - 1) / V::kRows;
  const int kv_items = (tokens * pg.kv_heads + V::kRows - 1) / V::kRows;
  for (int it = blockIdx.y * kWarps + warp; it < q_items + 2 * kv_items;
       it += gridDim.y * kWarps) {
    // queries, keys, values: uniform in a warp
    const int w = it < q_items ? 0 : it < q_items + kv_items ? 1 : 2;
    const int heads = w ? pg.kv_heads : p.H;
    const int row = (w == 0 ? it : it - q_items - (w - 1) * kv_items) * V::kRows + lane / V::kLanes;
    const int k = row < tokens * heads ? row / heads : 0;
    const int h = row - k * heads;
    const int pos = row < tokens * heads ? pos_of[k] : -1;
    const int64_t t = t0 + k;
    const __nv_bfloat16* x = (w == 0 ? p.q + t * p.qs : w == 1 ? p.k + t * p.ks : p.v + t * p.vs) +
                             static_cast<int64_t>(h) * D;
    __nv_bfloat16* y = w == 0 ? p.qo + (t * p.H + h) * D
                              : static_cast<__nv_bfloat16*>(w == 1 ? pg.K : pg.V) + row_at[k] +
                                    static_cast<int64_t>(h) * head_rows;
    Raw8<__nv_bfloat16> ra, rb;
    ra.zero();
    rb.zero();
    if (pos >= 0) {
      ra.load(x + at.a);
      rb.load(x + at.b);
    }
    if (w == 2) {
      if (pos < 0) continue;
      *reinterpret_cast<uint4*>(y + at.a) = ra.u;
      *reinterpret_cast<uint4*>(y + at.b) = rb.u;
      continue;
    }
    float2 a[4], b[4];
    ra.get(a);
    rb.get(b);
    Turns turns;
    turns.load(p.pe + static_cast<int64_t>(max(pos, 0)) * p.r, at.a, at.b, at.turns && pos >= 0,
               HALF);
    norm_rope_vec<D, HALF>(a, b, w == 0 ? p.gq : p.gk, at, turns, p.eps);
    // a bad entry: the query row is zeros, the page untouched
    if (pos == -1 || (w == 1 && pos < 0)) continue;
    if (pos < 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = b[i] = make_float2(0.f, 0.f);
    }
    store8(y + at.a, a);
    store8(y + at.b, b);
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

// Warps' shares of the work of the vector kernels: a warp takes all heads of
// its tokens, or, while that leaves fewer than eight warps to an SM, a part of
// their rounds.
struct VecShape {
  int64_t items;
  int parts;
};

VecShape vec_shape(int64_t tokens, int heads, int d) {
  const int groups = 512 / d;  // rows a warp has in flight
  const int64_t at_once = heads < groups && heads > 0 ? groups / heads : 1;
  const int64_t items = (tokens + at_once - 1) / at_once;
  const int rounds = (heads + groups - 1) / groups;
  const int64_t want = items > 0 ? 8 * static_cast<int64_t>(num_sms()) / items : 1;
  const int parts = want < 1 ? 1 : want < rounds ? static_cast<int>(want) : rounds < 1 ? 1 : rounds;
  return {items * parts, parts};
}

struct ForwardKernels {
  template <int D, typename T, int HALF>
  static constexpr auto get() { return norm_rope_vec_kernel<D, T, HALF>; }
};
struct BackwardKernels {
  template <int D, typename T, int HALF>
  static constexpr auto get() { return norm_rope_vec_bwd_kernel<D, T, HALF>; }
};

template <typename K, typename T>
void (*vec_kernel_of(int d, int half))(const TrainArgs, int) {
  if (d == 64) return half ? K::template get<64, T, 1>() : K::template get<64, T, 0>();
  return half ? K::template get<128, T, 1>() : K::template get<128, T, 0>();
}

template <typename K>
void (*vec_kernel(int d, int dtype, int half))(const TrainArgs, int) {
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
    const VecShape v = vec_shape(static_cast<int64_t>(B) * L, H + Hkv, d);
    vec_kernel<ForwardKernels>(d, dtype, pairing)<<<grid_for(v.items, 3), 32 * kWarps, 0, s>>>(
        p, v.parts);
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
  if (H + Hkv == 0 && !dgamma_q && !dgamma_k) return MHA_OK;
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
  if (bad_ptr(workspace, 16) || workspace_bytes < qk_norm_rope_backward_workspace_bytes(d))
    return MHA_ERR_INVALID_ARG;
  DeviceCtl ctl;
  if (!device_ctl(&ctl)) return MHA_ERR_CUDA;
  p.err = ctl.err;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t rows = static_cast<int64_t>(B) * L * (H > Hkv ? H : Hkv);
  const VecShape v = vec_shape(static_cast<int64_t>(B) * L, H > Hkv ? H : Hkv, d);
  unsigned blocks = rows == 0 ? 0 : vec ? grid_for(v.items, 2) : grid_for(rows, 4);
  if (blocks > kMaxGradBlocks) blocks = kMaxGradBlocks;
  if (blocks) {
    if (vec)
      vec_kernel<BackwardKernels>(d, dtype, pairing)<<<blocks, 32 * kWarps, 0, s>>>(p, v.parts);
    else if (dtype == MHA_BF16)
      norm_rope_any_bwd_kernel<__nv_bfloat16><<<blocks, 32 * kWarps, 0, s>>>(p);
    else
      norm_rope_any_bwd_kernel<float><<<blocks, 32 * kWarps, 0, s>>>(p);
  }
  // placed while the rows are still worked on, and waits for them
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((2 * d + 31) / 32);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, dgamma_kernel, static_cast<const float*>(p.partial),
                         static_cast<int>(blocks), d, dgamma[0], dgamma[1]) != cudaSuccess)
    return MHA_ERR_CUDA;
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
  // a round of rows for every warp, as long as the SMs have room
  const int token_blocks = (T + block_tokens - 1) / block_tokens;
  const int rounds = (H + 2 * Hkv + kWarps * (512 / d) - 1) / (kWarps * (512 / d));
  const int room = 2 * num_sms() / token_blocks;
  const dim3 grid(static_cast<unsigned>(token_blocks),
                  static_cast<unsigned>(room < 1 ? 1 : room < rounds ? room : rounds));
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
