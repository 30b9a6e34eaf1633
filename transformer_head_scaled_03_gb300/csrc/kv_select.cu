// kv_select.cu -- which pages of a long paged cache a query reads: the bounds
// of every full page's keys by columns, and for each new token and kv head the
// pages whose bounds admit the largest scores.
//
//   sum_c q_c k_c <= sum_c max(q_c lo_c, q_c hi_c)  where lo <= k <= hi
//                  = sum_c max(q_c, 0) hi_c + min(q_c, 0) lo_c
// With q, lo and hi in whole numbers of 8 bits the sum is exact (below 2^21),
// four products to an instruction, and two pages' rows of d bytes stand for
// 2 * page_size rows of keys and values.  Exact sums make the choice, and so
// the attention over it, the same for every order of summation.
#include <stdint.h>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kv_pages.cuh"
#include "ptx_cluster.cuh"
#include "ptx_pdl.cuh"

namespace mha {
namespace {

// The smallest power of two s >= 2^-100 with x <= 127 s; 0 for x = 0.  127 is
// 1.984375 * 2^6, so s is 2^(E - 6) for x = f * 2^E with f up to that.
__device__ __forceinline__ float step_of(float x) {
  if (x == 0.f) return 0.f;
  const unsigned u = __float_as_uint(x);
  int e = static_cast<int>(u >> 23) - 127 - 6 + ((u & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  e = max(e, -100);
  return __uint_as_float(static_cast<unsigned>(e + 127) << 23);
}

// ---------------------------------------------------------------------- bounds

struct BoundsArgs {
  PagesView pages;
  const int32_t* q_offsets;
  int T;
  int8_t* bounds;      // [num_pages, kv_heads, 2, d]
  float* bound_scale;  // [num_pages, kv_heads]
  unsigned* err;
};

constexpr int kBoundWarps = 8;

// Which full page unit u is: pages are numbered sequence by sequence, a warp
// summing up 32 sequences at a time.  False behind the last.
__device__ __forceinline__ bool full_page_of(const BoundsArgs& a, int64_t u, bool report, int* b_out,
                                             int* col) {
  const int lane = threadIdx.x & 31;
  const PagesView& pg = a.pages;
  int64_t rest = u;
  for (int b0 = 0; b0 < pg.B; b0 += 32) {
    const int b = b0 + lane;
    int first = 0, count = 0;
    if (b < pg.B) {
      const int q0 = __ldg(a.q_offsets + b), q1 = __ldg(a.q_offsets + b + 1);
      const int len = __ldg(pg.kv_len + b), n = q1 - q0;
      const bool bad = q0 < 0 || q1 < q0 || q1 > a.T ||
                       (n > 0 && (len < n || len > (static_cast<int64_t>(pg.cols) << pg.page_shift)));
      if (bad && report) atomicOr(a.err, kErrPages);
      if (!bad && n > 0) {
        first = (len - n) >> pg.page_shift;
        count = (len >> pg.page_shift) - first;
      }
    }
    int64_t incl = count;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, incl, s);
      if (lane >= s) incl += up;
    }
    const unsigned in = __ballot_sync(0xffffffffu, rest < incl);
    if (in) {
      const int src = __ffs(in) - 1;
      *b_out = b0 + src;
      *col = static_cast<int>(__shfl_sync(0xffffffffu, rest - (incl - count) + first, src));
      return true;
    }
    rest -= __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

// 16 bytes of keys as minima and maxima.
template <bool E8>
struct Extremes;

template <>
struct Extremes<false> {
  __nv_bfloat162 lo[4], hi[4];
  __device__ __forceinline__ void set(uint4 u) {
    const __nv_bfloat162* v = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) lo[i] = hi[i] = v[i];
  }
  __device__ __forceinline__ void add(uint4 u) {
    const __nv_bfloat162* v = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) lo[i] = __hmin2(lo[i], v[i]), hi[i] = __hmax2(hi[i], v[i]);
  }
  __device__ __forceinline__ void exchange(int mask) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = __hmin2(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], mask));
      hi[i] = __hmax2(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], mask));
    }
  }
  static constexpr int kCols = 8;
  __device__ __forceinline__ void get(float (&l)[8], float (&h)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = __bfloat1622float2(lo[i]), b = __bfloat1622float2(hi[i]);
      l[2 * i] = a.x, l[2 * i + 1] = a.y, h[2 * i] = b.x, h[2 * i + 1] = b.y;
    }
  }
};

// Codes as the high bytes of bf16 numbers, whose order is theirs (no code's bits
// there are an infinity or a NaN): two to an instruction, where decoding them
// first would wait for the conversion unit.
template <>
struct Extremes<true> {
  __nv_bfloat162 lo[8], hi[8];
  static __device__ __forceinline__ __nv_bfloat162 two(unsigned w, int odd) {
    const unsigned x = odd ? w & 0xff00ff00u : w << 8 & 0xff00ff00u;
    return *reinterpret_cast<const __nv_bfloat162*>(&x);
  }
  __device__ __forceinline__ void set(uint4 u) {
    const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) lo[i] = hi[i] = two(w[i / 2], i & 1);
  }
  __device__ __forceinline__ void add(uint4 u) {
    const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 v = two(w[i / 2], i & 1);
      lo[i] = __hmin2(lo[i], v), hi[i] = __hmax2(hi[i], v);
    }
  }
  __device__ __forceinline__ void exchange(int mask) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] = __hmin2(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], mask));
      hi[i] = __hmax2(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], mask));
    }
  }
  static constexpr int kCols = 16;
  // (even columns' codes lie in element 2 k of a word, odd ones' in 2 k + 1)
  __device__ __forceinline__ void get(float (&l)[16], float (&h)[16]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = 4 * (i / 2) + (i & 1);
      decode(lo[i], l[c], l[c + 2]);
      decode(hi[i], h[c], h[c + 2]);
    }
  }
  static __device__ __forceinline__ void decode(__nv_bfloat162 v, float& a, float& b) {
    const unsigned x = *reinterpret_cast<const unsigned*>(&v);
    const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((x >> 8 & 0xffu) | (x >> 16 & 0xff00u)), __NV_E4M3)));
    a = f.x, b = f.y;
  }
};

// A warp per (full page, kv head): the page's rows of a head lie one behind
// the other, so a lane's 16 bytes keep their columns from load to load.
template <int D, bool E8>
__global__ void __launch_bounds__(32 * kBoundWarps) kv_bounds_kernel(const BoundsArgs a) {
  const PagesView& pg = a.pages;
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kBoundWarps + (threadIdx.x >> 5);
  int b = 0, col = 0;
  // the first warp of all looks at every sequence for its report
  if (unit == 0) full_page_of(a, int64_t{1} << 40, true, &b, &col);
  if (!full_page_of(a, unit / pg.kv_heads, false, &b, &col)) return;
  const int g = static_cast<int>(unit % pg.kv_heads);
  const int page = __ldg(pg.table + static_cast<int64_t>(b) * pg.cols + col);
  if (page < 0 || page >= pg.num_pages) {
    if (lane == 0) atomicOr(a.err, kErrPages);
    return;
  }
  constexpr int kEs = E8 ? 1 : 2;
  constexpr int kRowVecs = D * kEs / 16;  // lanes to a row
  const uint4* from = reinterpret_cast<const uint4*>(
      static_cast<const char*>(pg.K) +
      (page * pg.page_stride + ((static_cast<int64_t>(g) * D) << pg.page_shift)) * kEs);
  const int vecs = kRowVecs << pg.page_shift;  // a multiple of 32
  Extremes<E8> x;
  x.set(__ldg(from + lane));
#pragma unroll 4
  for (int v = 32 + lane; v < vecs; v += 32) x.add(__ldg(from + v));
#pragma unroll
  for (int s = kRowVecs; s < 32; s <<= 1) x.exchange(s);
  constexpr int N = Extremes<E8>::kCols;
  float lo[N], hi[N];
  x.get(lo, hi);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, fmaxf(-lo[i], hi[i]));
  const float step = step_of(warp_max_f32(top));
  // a power of two: the products are exact
  const float inv = step > 0.f ? __uint_as_float(0x7f000000u - __float_as_uint(step)) : 0.f;
  if (lane < kRowVecs) {
    uint32_t l4[N / 4], h4[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      l4[i] = h4[i] = 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int il = __float2int_rd(lo[4 * i + k] * inv), ih = __float2int_ru(hi[4 * i + k] * inv);
        l4[i] |= (static_cast<unsigned>(il) & 0xffu) << (8 * k);
        h4[i] |= (static_cast<unsigned>(ih) & 0xffu) << (8 * k);
      }
    }
    const int64_t at = static_cast<int64_t>(page) * pg.kv_heads + g;
    uint32_t* out = reinterpret_cast<uint32_t*>(a.bounds + at * 2 * D + lane * N);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      out[i] = l4[i];
      out[D / 4 + i] = h4[i];
    }
    if (lane == 0) a.bound_scale[at] = E8 ? step * pg.k_scale[at] : step;
  }
}

// ---------------------------------------------------------------------- scores

struct SelectArgs {
  const __nv_bfloat16* q;
  int64_t qs;
  PagesView pages;  // K, V and strides are not used
  const int32_t* q_offsets;
  const int8_t* bounds;
  const float* bound_scale;
  int T, H, G, n_select;
  int32_t* selected;
  int32_t* lengths;
  float* scores;  // [T, kv_heads, cols]
  unsigned* err;
};

// A token's sequence and position; state 0: no sequence's, -1: a bad entry.
struct TokenPlace {
  int b, pos, state;
};

__device__ __forceinline__ TokenPlace place_of(const SelectArgs& a, int t) {
  const PagesView& pg = a.pages;
  TokenPlace w{sequence_of_token(a.q_offsets, pg.B, t), 0, 0};
  if (w.b >= pg.B) return w;
  const int q0 = __ldg(a.q_offsets + w.b), q1 = __ldg(a.q_offsets + w.b + 1);
  const int len = __ldg(pg.kv_len + w.b);
  if (q0 < 0 || q1 < q0 || q1 > a.T || t >= q1 || (w.b > 0 && t < q0)) {
    w.state = -1;
  } else if (t >= q0) {
    const int n = q1 - q0;
    w.pos = len - n + (t - q0);
    w.state = len >= n && len <= (static_cast<int64_t>(pg.cols) << pg.page_shift) ? 1 : -1;
  }
  return w;
}

constexpr int kScoreWarps = 4;
constexpr int kRun = 32;          // pages of a warp: one look-up of their numbers
constexpr int kHeadsAtOnce = 16;  // query heads in shared memory at a time
// the score that marks a bad page number (a NaN no product gives)
constexpr unsigned kBadScore = 0x7fffffffu;

__device__ __forceinline__ int dot16(uint4 q, uint4 x, int s) {
  s = __dp4a(static_cast<int>(q.x), static_cast<int>(x.x), s);
  s = __dp4a(static_cast<int>(q.y), static_cast<int>(x.y), s);
  s = __dp4a(static_cast<int>(q.z), static_cast<int>(x.z), s);
  return __dp4a(static_cast<int>(q.w), static_cast<int>(x.w), s);
}

// The scores of one (token, kv head)'s pages, a run of kRun neighbouring ones to
// a warp: D / 16 lanes to a page, 16 columns of lo and hi to a lane, kAhead
// rounds of pages under way.  Four heads' sums are spread over the lanes while
// they are summed up, half as many exchanges as one by one.
template <int D>
__global__ void __launch_bounds__(32 * kScoreWarps)
    kv_score_kernel(const SelectArgs a, int chunks) {
  constexpr int L = D / 16;       // lanes per page
  constexpr int kPages = 32 / L;  // pages per warp and round
  constexpr int kAhead = 4;
  static_assert(kRun % (kPages * kAhead) == 0, "whole rounds");
  __shared__ uint4 q_pos[kHeadsAtOnce][L], q_neg[kHeadsAtOnce][L];
  __shared__ float q_step[kHeadsAtOnce];
  const PagesView& pg = a.pages;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int item = static_cast<int>(blockIdx.x / static_cast<unsigned>(chunks));
  const int chunk = static_cast<int>(blockIdx.x % static_cast<unsigned>(chunks));
  const int t = item / pg.kv_heads, g = item % pg.kv_heads;
  pdl_launch_dependents();
  const TokenPlace w = place_of(a, t);
  const int newest = w.pos >> pg.page_shift;  // full pages that the token sees
  const int b0 = chunk * kScoreWarps * kRun;
  // without a choice to make, or pages of this stretch, there is nothing to score
  if (w.state < 1 || newest < a.n_select || b0 >= newest) return;
  const int c0 = b0 + warp * kRun;
  int pages = -1;
  if (c0 + lane < newest) pages = __ldg(pg.table + static_cast<int64_t>(w.b) * pg.cols + c0 + lane);
  const bool good = pages >= 0 && pages < pg.num_pages;
  const int64_t at0 = static_cast<int64_t>(good ? pages : 0) * pg.kv_heads + g;
  float scale = 0.f;
  if (good) scale = __ldg(a.bound_scale + at0);
  const int part = lane % L;
  // this lane's heads of four, after the sums
  const int mine = (lane & L / 2 ? 2 : 0) + (lane & L / 4 ? 1 : 0);
  float best[kRun / kPages];
#pragma unroll
  for (int i = 0; i < kRun / kPages; ++i) best[i] = -INFINITY;
  for (int h0 = 0; h0 < a.G; h0 += kHeadsAtOnce) {
    const int heads = min(kHeadsAtOnce, a.G - h0);
    if (h0) __syncthreads();
    // a warp rounds a query row: D / 32 neighbouring columns to a lane
    for (int h = warp; h < heads; h += kScoreWarps) {
      constexpr int N = D / 32;
      const __nv_bfloat16* q =
          a.q + t * a.qs + static_cast<int64_t>(g * a.G + h0 + h) * D + lane * N;
      float x[N];
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        x[i] = __bfloat162float(q[i]);
        if (!isfinite(x[i])) x[i] = 0.f;
        top = fmaxf(top, fabsf(x[i]));
      }
      const float step = step_of(warp_max_f32(top));
      const float inv = step > 0.f ? __uint_as_float(0x7f000000u - __float_as_uint(step)) : 0.f;
      int8_t* up = reinterpret_cast<int8_t*>(q_pos[h]) + lane * N;
      int8_t* un = reinterpret_cast<int8_t*>(q_neg[h]) + lane * N;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int v = __float2int_rn(x[i] * inv);
        up[i] = static_cast<int8_t>(max(v, 0));
        un[i] = static_cast<int8_t>(min(v, 0));
      }
      if (lane == 0) q_step[h] = step;
    }
    __syncthreads();
#pragma unroll
    for (int i0 = 0; i0 < kRun / kPages; i0 += kAhead) {
      if (c0 + i0 * kPages >= newest) break;
      uint4 lo[kAhead], hi[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        // a page behind the last, or a bad one, reads page 0's: nothing comes of it
        const int64_t at = __shfl_sync(0xffffffffu, at0, (i0 + i) * kPages + lane / L);
        const uint4* from = reinterpret_cast<const uint4*>(a.bounds + at * 2 * D) + part;
        lo[i] = __ldg(from);
        hi[i] = __ldg(from + L);
      }
      for (int h = 0; h < heads; h += 4) {
        int s[kAhead][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // heads behind the last are the last once more
          const int hk = min(h + k, heads - 1);
          const uint4 qp = q_pos[hk][part], qn = q_neg[hk][part];
#pragma unroll
          for (int i = 0; i < kAhead; ++i) s[i][k] = dot16(qn, lo[i], dot16(qp, hi[i], 0));
        }
        const float step = q_step[min(h + mine, heads - 1)];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const bool upper = lane & L / 2, second = lane & L / 4;
          int a0 = upper ? s[i][2] : s[i][0], a1 = upper ? s[i][3] : s[i][1];
          a0 += __shfl_xor_sync(0xffffffffu, upper ? s[i][0] : s[i][2], L / 2);
          a1 += __shfl_xor_sync(0xffffffffu, upper ? s[i][1] : s[i][3], L / 2);
          int sum = (second ? a1 : a0) + __shfl_xor_sync(0xffffffffu, second ? a0 : a1, L / 4);
#pragma unroll
          for (int k = L / 8; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
          best[i0 + i] = fmaxf(best[i0 + i], static_cast<float>(sum) * step);
        }
      }
    }
  }
  // page l of the run to lane l, coalesced
  float score = 0.f;
#pragma unroll
  for (int i = 0; i < kRun / kPages; ++i) {
    float x = best[i];
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, L / 2));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, L / 4));
    const float v = __shfl_sync(0xffffffffu, x, lane % kPages * L);
    if (lane / kPages == i) score = v;
  }
  // + 0: a product that underflows has no sign
  score = score * scale + 0.f;
  if (c0 + lane < newest)
    a.scores[(static_cast<int64_t>(t) * pg.kv_heads + g) * pg.cols + c0 + lane] =
        good ? score : __uint_as_float(kBadScore);
}

// --------------------------------------------------------------------- choice

constexpr int kPickThreads = 512;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kPickKeys = 8192;  // that stay in shared memory; those behind are read again

// fp32 in the order of unsigned whole numbers; a NaN, which finite bounds and
// scales never give, below all others.
__device__ __forceinline__ unsigned rank_key(float x) {
  const unsigned u = __float_as_uint(x);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One block per (token, kv head): the n_select - 1 largest scores by a search
// for the smallest of them, eight bits at a time from the highest one in which
// any two differ (scores share their exponent's first bits, and one bin's
// counter would serialise them), then the pages in order.
__global__ void __launch_bounds__(kPickThreads) kv_pick_kernel(const SelectArgs a) {
  __shared__ unsigned keys[kPickKeys];
  __shared__ int bins[256];
  __shared__ int counts[2][kPickWarps];
  __shared__ unsigned least[kPickWarps], most[kPickWarps];
  __shared__ int found[2];
  const PagesView& pg = a.pages;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x / pg.kv_heads, g = blockIdx.x % pg.kv_heads;
  const TokenPlace w = place_of(a, t);
  const int newest = w.pos >> pg.page_shift;
  const int32_t* row = pg.table + static_cast<int64_t>(w.b) * pg.cols;
  int32_t* out = a.selected + (static_cast<int64_t>(t) * pg.kv_heads + g) * a.n_select;
  const float* scores = a.scores + (static_cast<int64_t>(t) * pg.kv_heads + g) * pg.cols;
  int picked = 0;
  bool bad = w.state < 0;
  for (int i = threadIdx.x; i < 256; i += kPickThreads) bins[i] = 0;
  pdl_wait();
  if (w.state == 1 && newest < a.n_select) {
    // every page there is
    bool wrong = false;
    for (int c = threadIdx.x; c <= newest; c += kPickThreads) {
      const int page = __ldg(row + c);
      wrong = wrong || page < 0 || page >= pg.num_pages;
      out[c] = page;
    }
    bad = __syncthreads_or(wrong);
    picked = newest + 1;
  } else if (w.state == 1) {
    const int want = a.n_select - 1;
    bool wrong = false;
    unsigned lo = 0xffffffffu, hi = 0u;
    for (int c = threadIdx.x; c < newest; c += kPickThreads) {
      const float x = scores[c];
      const unsigned key = rank_key(x);
      wrong = wrong || __float_as_uint(x) == kBadScore;
      if (c < kPickKeys) keys[c] = key;
      lo = min(lo, key);
      hi = max(hi, key);
    }
    auto key_of = [&](int c) { return c < kPickKeys ? keys[c] : rank_key(scores[c]); };
    if (threadIdx.x == 0) {
      const int page = __ldg(row + newest);
      wrong = wrong || page < 0 || page >= pg.num_pages;
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
      least[warp] = lo;
      most[warp] = hi;
    }
    bad = __syncthreads_or(wrong);
#pragma unroll
    for (int i = 0; i < kPickWarps; ++i) {
      lo = min(lo, least[i]);
      hi = max(hi, most[i]);
    }
    // the want-th largest key, and how many of the equal ones are in.  Above
    // bit `top` all keys agree.
    int top = lo == hi ? 0 : 32 - __clz(lo ^ hi);
    unsigned prefix = top == 32 ? 0u : hi >> top << top;
    int left = want;
    while (top > 0 && want > 0) {
      const int shift = max(top - 8, 0);
      for (int c = threadIdx.x; c < newest; c += kPickThreads) {
        const unsigned key = key_of(c);
        if (top == 32 || key >> top == prefix >> top)
          atomicAdd(&bins[(key >> shift) & (0xffu >> (8 - (top - shift)))], 1);
      }
      __syncthreads();
      if (warp == 0) {
        // lane l: bins 255 - 8 l and the seven below
        int mine[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sum += mine[i] = bins[255 - 8 * lane - i];
          bins[255 - 8 * lane - i] = 0;
        }
        int incl = sum;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
          const int up = __shfl_up_sync(0xffffffffu, incl, s);
          if (lane >= s) incl += up;
        }
        int before = incl - sum;
        if (before < left && incl >= left) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (before < left && before + mine[i] >= left) {
              found[0] = 255 - 8 * lane - i;
              found[1] = left - before;
            }
            before += mine[i];
          }
        }
      }
      __syncthreads();
      prefix |= static_cast<unsigned>(found[0]) << shift;
      left = found[1];
      top = shift;
    }
    // a warp takes a stretch of neighbouring columns: first its number of
    // larger and of equal keys, then the places
    const int stretch = (newest + kPickThreads - 1) / kPickThreads * 32;
    const int s0 = warp * stretch, s1 = min(newest, s0 + stretch);
    int above = 0, equal = 0;
    for (int c = s0 + lane; c - lane < s1; c += 32) {
      const unsigned key = c < s1 ? key_of(c) : 0u;
      above += __popc(__ballot_sync(0xffffffffu, c < s1 && want > 0 && key > prefix));
      equal += __popc(__ballot_sync(0xffffffffu, c < s1 && want > 0 && key == prefix));
    }
    if (lane == 0) {
      counts[0][warp] = above;
      counts[1][warp] = equal;
    }
    __syncthreads();
    int a0 = 0, e0 = 0;  // of the warps before
    for (int i = 0; i < warp; ++i) {
      a0 += counts[0][i];
      e0 += counts[1][i];
    }
    for (int c = s0 + lane; c - lane < s1; c += 32) {
      const unsigned key = c < s1 ? key_of(c) : 0u;
      const bool is_above = c < s1 && want > 0 && key > prefix;
      const bool is_equal = c < s1 && want > 0 && key == prefix;
      const unsigned ma = __ballot_sync(0xffffffffu, is_above);
      const unsigned me = __ballot_sync(0xffffffffu, is_equal);
      const unsigned below = (1u << lane) - 1u;
      const int na = a0 + __popc(ma & below), ne = e0 + __popc(me & below);
      // of the equal ones before this column, at most `left` are in
      if (is_above || (is_equal && ne < left)) out[na + min(ne, left)] = __ldg(row + c);
      a0 += __popc(ma);
      e0 += __popc(me);
    }
    if (threadIdx.x == 0) out[want] = __ldg(row + newest);
    picked = a.n_select;
  }
  if (bad) {
    if (threadIdx.x == 0) atomicOr(a.err, kErrPages);
    __syncthreads();
    picked = 0;
  }
  for (int i = picked + threadIdx.x; i < a.n_select; i += kPickThreads) out[i] = -1;
  if (g == 0 && threadIdx.x == 0)
    a.lengths[t] = bad ? -1
                   : w.state == 0
                       ? 0
                       : ((min(newest + 1, a.n_select) - 1) << pg.page_shift) +
                             (w.pos & ((1 << pg.page_shift) - 1)) + 1;
}

bool bad_ptr(const void* p, uintptr_t align) {
  return !p || (reinterpret_cast<uintptr_t>(p) & (align - 1));
}

}  // namespace
}  // namespace mha

using namespace mha;

extern "C" {

mha_status kv_pages_bounds(const mha_kv_pages* pages, const mha_kv_scales* scales, int layer,
                           const int32_t* q_offsets, int T, int8_t* bounds, float* bound_scale,
                           mha_stream stream) {
  const mha_status st = validate_pages_any(pages, scales);
  if (st != MHA_OK) return st;
  if (T < 0 || layer < 0 || layer >= pages->layers) return MHA_ERR_INVALID_ARG;
  const int d = pages->d;
  if (pages->dtype == MHA_F32 || (d != 64 && d != 128)) return MHA_ERR_UNSUPPORTED;
  if (T == 0 || pages->B == 0) return MHA_OK;
  if (bad_ptr(q_offsets, 4) || bad_ptr(bounds, 16) || bad_ptr(bound_scale, 4))
    return MHA_ERR_INVALID_ARG;
  DeviceCtl ctl;
  if (!device_ctl(&ctl)) return MHA_ERR_CUDA;
  const int64_t at = static_cast<int64_t>(pages->num_pages) * pages->kv_heads * layer;
  const BoundsArgs a{pages_view(*pages, layer, scales), q_offsets, T, bounds + at * 2 * d,
                     bound_scale + at, ctl.err};
  // pages that T tokens can have filled: one for every page_size of a
  // sequence's, and one more
  const int64_t seqs = T < pages->B ? T : pages->B;
  const int64_t full = T / pages->page_size + seqs;
  const int64_t units = (full < T ? full : T) * pages->kv_heads;
  const int64_t blocks = (units + kBoundWarps - 1) / kBoundWarps;
  if (blocks > 0x7fffffffLL) return MHA_ERR_UNSUPPORTED;
  const unsigned n = static_cast<unsigned>(blocks);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d == 64 && scales)
    kv_bounds_kernel<64, true><<<n, 32 * kBoundWarps, 0, s>>>(a);
  else if (d == 64)
    kv_bounds_kernel<64, false><<<n, 32 * kBoundWarps, 0, s>>>(a);
  else if (scales)
    kv_bounds_kernel<128, true><<<n, 32 * kBoundWarps, 0, s>>>(a);
  else
    kv_bounds_kernel<128, false><<<n, 32 * kBoundWarps, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? MHA_OK : MHA_ERR_CUDA;
}

size_t kv_pages_select_workspace_bytes(int T, int kv_heads, int table_cols) {
  if (T < 0 || kv_heads < 1 || table_cols < 1) return 0;
  return static_cast<size_t>(T) * kv_heads * table_cols * sizeof(float);
}

mha_status kv_pages_select(const void* Q, int64_t q_token_stride, const mha_kv_pages* pages,
                           int layer, const int32_t* q_offsets, const int8_t* bounds,
                           const float* bound_scale, int T, int H, int n_select,
                           int32_t* selected, int32_t* lengths, void* workspace,
                           size_t workspace_bytes, mha_stream stream) {
  const mha_status st = validate_pages_shape(pages);
  if (st != MHA_OK) return st;
  if (T < 0 || H < 1 || n_select < 1 || layer < 0 || layer >= pages->layers ||
      H % pages->kv_heads != 0)
    return MHA_ERR_INVALID_ARG;
  const int d = pages->d, Hkv = pages->kv_heads, G = H / Hkv;
  if (q_token_stride == 0) q_token_stride = static_cast<int64_t>(H) * d;
  if (q_token_stride < static_cast<int64_t>(H) * d) return MHA_ERR_INVALID_ARG;
  if (pages->dtype == MHA_F32 || (d != 64 && d != 128) || G > 128 || n_select > 65536)
    return MHA_ERR_UNSUPPORTED;
  if (T == 0) return MHA_OK;
  if (bad_ptr(Q, 2) || bad_ptr(bounds, 16) || bad_ptr(bound_scale, 4) || bad_ptr(selected, 4) ||
      bad_ptr(lengths, 4) || (pages->B > 0 && bad_ptr(q_offsets, 4)) || bad_ptr(workspace, 16) ||
      workspace_bytes < kv_pages_select_workspace_bytes(T, Hkv, pages->table_cols))
    return MHA_ERR_INVALID_ARG;
  const int64_t items = static_cast<int64_t>(T) * Hkv;
  DeviceCtl ctl;
  if (!device_ctl(&ctl)) return MHA_ERR_CUDA;
  const int64_t at = static_cast<int64_t>(pages->num_pages) * Hkv * layer;
  const SelectArgs a{static_cast<const __nv_bfloat16*>(Q), q_token_stride, pages_view(*pages, layer),
                     q_offsets, bounds + at * 2 * d, bound_scale + at, T, H, G, n_select, selected,
                     lengths, static_cast<float*>(workspace), ctl.err};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int chunks = (pages->table_cols + kScoreWarps * kRun - 1) / (kScoreWarps * kRun);
  const int64_t blocks = items * chunks;
  if (blocks > 0x7fffffffLL) return MHA_ERR_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>(blocks);
  if (d == 64)
    kv_score_kernel<64><<<grid, 32 * kScoreWarps, 0, s>>>(a, chunks);
  else
    kv_score_kernel<128><<<grid, 32 * kScoreWarps, 0, s>>>(a, chunks);
  if (cudaGetLastError() != cudaSuccess) return MHA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items));
  cfg.blockDim = dim3(kPickThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kv_pick_kernel, a) != cudaSuccess) return MHA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MHA_OK : MHA_ERR_CUDA;
}

}  // extern "C"
