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
//
// Bound by latency: a few dependent look-ups, then one round of loads.  Measured
// (32 query heads on 8 kv heads, d = 128), in a graph: bounds of 2,250 pages of 32
// rows in 8 bits 20 us (78 MB, 3.9 TB/s), of the few that a decoding step fills 3
// us; 64 of 2,048 pages chosen for one token 8.6 us; 128 of 2,048 to 4,096 for 16
// tokens 30 us (the scores read 100 MB; 25 us of them under a profiler).
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

// Whether a sequence's offsets are bad, or its length for the new tokens they say.
__device__ __forceinline__ bool bad_sequence(const PagesView& pg, int T, int q0, int q1, int len) {
  const int n = q1 - q0;
  return q0 < 0 || q1 < q0 || q1 > T ||
         (n > 0 && (len < n || len > (static_cast<int64_t>(pg.cols) << pg.page_shift)));
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

// Which full page `rest` of them is: pages are numbered sequence by sequence, a
// warp summing up 32 sequences at a time.  False behind the last.
__device__ __forceinline__ bool full_page_of(const BoundsArgs& a, int rest, bool report, int* b_out,
                                             int* col) {
  const int lane = threadIdx.x & 31;
  const PagesView& pg = a.pages;
  for (int b0 = 0; b0 < pg.B; b0 += 32) {
    const int b = b0 + lane;
    int first = 0, count = 0;
    if (b < pg.B) {
      const int q0 = __ldg(a.q_offsets + b), q1 = __ldg(a.q_offsets + b + 1);
      const int len = __ldg(pg.kv_len + b), n = q1 - q0;
      const bool bad = bad_sequence(pg, a.T, q0, q1, len);
      if (bad && report) atomicOr(a.err, kErrPages);
      if (!bad && n > 0) {
        first = (len - n) >> pg.page_shift;
        count = (len >> pg.page_shift) - first;
      }
    }
    // at most 32 sequences of 2^26 pages
    unsigned incl = static_cast<unsigned>(count);
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const unsigned up = __shfl_up_sync(0xffffffffu, incl, s);
      if (lane >= s) incl += up;
    }
    const unsigned in = __ballot_sync(0xffffffffu, static_cast<unsigned>(rest) < incl);
    if (in && !report) {
      const int src = __ffs(in) - 1;
      *b_out = b0 + src;
      *col = __shfl_sync(0xffffffffu, rest - static_cast<int>(incl) + count + first, src);
      return true;
    }
    rest -= static_cast<int>(__shfl_sync(0xffffffffu, incl, 31));
    if (rest < 0) rest = 0;  // of a report
  }
  return false;
}

// 16 bytes of keys as numbers in bf16, two to a register: bf16 as it is; codes as
// the high bytes of bf16 numbers, whose order is theirs (no code's bits there
// are an infinity or a NaN), where decoding them first would wait for the
// conversion unit.
template <bool E8>
struct Keys16 {
  static constexpr int kRegs = E8 ? 8 : 4;
  static __device__ __forceinline__ __nv_bfloat162 at(const uint4& u, int i) {
    const unsigned w[4] = {u.x, u.y, u.z, u.w};
    const unsigned x = !E8 ? w[i & 3] : i & 1 ? w[i / 2] & 0xff00ff00u : w[i / 2] << 8 & 0xff00ff00u;
    return *reinterpret_cast<const __nv_bfloat162*>(&x);
  }
  // The first column of register i; the other is the next, of codes the one
  // after that.
  static __device__ __forceinline__ int column(int i) { return E8 ? 4 * (i / 2) + (i & 1) : 2 * i; }
  static __device__ __forceinline__ float2 values(__nv_bfloat162 v) {
    if constexpr (!E8) return __bfloat1622float2(v);
    const unsigned x = *reinterpret_cast<const unsigned*>(&v);
    return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((x >> 8 & 0xffu) | (x >> 16 & 0xff00u)), __NV_E4M3)));
  }
};

// N registers of minima and maxima down to `R`, over the lanes that hold other
// rows of the same columns: each exchange halves the registers of a lane.  at0
// becomes the place of those that are left.
template <int N, int R>
__device__ __forceinline__ void reduce_rows(__nv_bfloat162 (&lo)[N], __nv_bfloat162 (&hi)[N],
                                            int& at0) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = N / 2, mask = 16; n >= R; n /= 2, mask /= 2) {
    const bool upper = lane & mask;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if (i >= n) break;
      const __nv_bfloat162 gl = upper ? lo[i] : lo[n + i], gh = upper ? hi[i] : hi[n + i];
      const __nv_bfloat162 kl = upper ? lo[n + i] : lo[i], kh = upper ? hi[n + i] : hi[i];
      lo[i] = __hmin2(kl, __shfl_xor_sync(0xffffffffu, gl, mask));
      hi[i] = __hmax2(kh, __shfl_xor_sync(0xffffffffu, gh, mask));
    }
    at0 += upper ? n : 0;
  }
}

// A warp per (full page, kv head): the page's rows of a head lie one behind the
// other, so a lane's 16 bytes keep their columns from load to load.
template <int D, bool E8>
__global__ void __launch_bounds__(32 * kBoundWarps) kv_bounds_kernel(const BoundsArgs a) {
  using K = Keys16<E8>;
  const PagesView& pg = a.pages;
  const int lane = threadIdx.x & 31;
  const unsigned unit = blockIdx.x * kBoundWarps + (threadIdx.x >> 5);
  int b = 0, col = 0;
  // the first warp of all looks at every sequence for its report
  if (unit == 0) full_page_of(a, 0, true, &b, &col);
  if (!full_page_of(a, static_cast<int>(unit / pg.kv_heads), false, &b, &col)) return;
  const int g = static_cast<int>(unit % pg.kv_heads);
  const int page = __ldg(pg.table + static_cast<int64_t>(b) * pg.cols + col);
  if (page < 0 || page >= pg.num_pages) {
    if (lane == 0) atomicOr(a.err, kErrPages);
    return;
  }
  constexpr int kEs = E8 ? 1 : 2;
  constexpr int kRowVecs = D * kEs / 16;        // lanes to a row
  constexpr int kRegs = K::kRegs;
  constexpr int kLeft = kRegs * kRowVecs / 32;  // registers of a lane in the end
  static_assert(kLeft == 1 || kLeft == 2, "a lane's columns");
  const uint4* from = reinterpret_cast<const uint4*>(
      static_cast<const char*>(pg.K) +
      (page * pg.page_stride + ((static_cast<int64_t>(g) * D) << pg.page_shift)) * kEs) + lane;
  const int vecs = kRowVecs << pg.page_shift;  // a multiple of 32
  const int64_t at = static_cast<int64_t>(page) * pg.kv_heads + g;
  const float page_scale = E8 ? __ldg(pg.k_scale + at) : 1.f;
  __nv_bfloat162 lo[kRegs], hi[kRegs];
  constexpr int kAtOnce = 4;
  for (int v = 0; v < vecs; v += 32 * kAtOnce) {
    uint4 u[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      if (v + 32 * k < vecs) u[k] = __ldg(from + v + 32 * k);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (v + 32 * k >= vecs) break;
#pragma unroll
      for (int i = 0; i < kRegs; ++i) {
        const __nv_bfloat162 x = K::at(u[k], i);
        lo[i] = v + k == 0 ? x : __hmin2(lo[i], x);
        hi[i] = v + k == 0 ? x : __hmax2(hi[i], x);
      }
    }
  }
  int at0 = 0;
  reduce_rows<kRegs, kLeft>(lo, hi, at0);
  float2 l[kLeft], h[kLeft];
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kLeft; ++i) {
    l[i] = K::values(lo[i]);
    h[i] = K::values(hi[i]);
    top = fmaxf(top, fmaxf(fmaxf(-l[i].x, -l[i].y), fmaxf(h[i].x, h[i].y)));
  }
  const float step = step_of(warp_max_f32(top));
  // a power of two: the products are exact
  const float inv = step > 0.f ? __uint_as_float(0x7f000000u - __float_as_uint(step)) : 0.f;
  int8_t* out = a.bounds + at * 2 * D + lane % kRowVecs * (16 / kEs);
#pragma unroll
  for (int i = 0; i < kLeft; ++i) {
    const int c = K::column(at0 + i), next = E8 ? 2 : 1;
    out[c] = static_cast<int8_t>(__float2int_rd(l[i].x * inv));
    out[c + next] = static_cast<int8_t>(__float2int_rd(l[i].y * inv));
    out[D + c] = static_cast<int8_t>(__float2int_ru(h[i].x * inv));
    out[D + c + next] = static_cast<int8_t>(__float2int_ru(h[i].y * inv));
  }
  if (lane == 0) a.bound_scale[at] = E8 ? step * page_scale : step;
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

// The sequence is the first whose tokens end behind t; 32 of them are looked at
// with one round of loads.  Warp-collective.
__device__ __forceinline__ TokenPlace place_of(const SelectArgs& a, int t) {
  const PagesView& pg = a.pages;
  const int lane = threadIdx.x & 31;
  for (int b0 = 0; b0 < pg.B; b0 += 32) {
    const int b = b0 + lane;
    int q0 = 0, q1 = 0, len = 0;
    if (b < pg.B) {
      q0 = __ldg(a.q_offsets + b);
      q1 = __ldg(a.q_offsets + b + 1);
      len = __ldg(pg.kv_len + b);
    }
    const unsigned behind = __ballot_sync(0xffffffffu, b < pg.B && q1 > t);
    if (!behind) continue;
    const int src = __ffs(behind) - 1;
    q0 = __shfl_sync(0xffffffffu, q0, src);
    q1 = __shfl_sync(0xffffffffu, q1, src);
    len = __shfl_sync(0xffffffffu, len, src);
    TokenPlace w{b0 + src, 0, 0};
    if (q0 < 0 || q1 < q0 || q1 > a.T || (w.b > 0 && t < q0)) {
      w.state = -1;
    } else if (t >= q0) {
      const int n = q1 - q0;
      w.pos = len - n + (t - q0);
      w.state = len >= n && len <= (static_cast<int64_t>(pg.cols) << pg.page_shift) ? 1 : -1;
    }
    if (w.state < 1) w.pos = 0;
    return w;
  }
  return TokenPlace{0, 0, 0};
}

constexpr int kScoreWarps = 4;
constexpr int kHeadsAtOnce = 16;  // query heads in shared memory at a time
// the score that marks a bad page number (a NaN that no product gives: theirs is
// 0x7fffffff)
constexpr unsigned kBadScore = 0xffc00001u;

// 16 bytes from global to shared memory, not waited for.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ int dot16(uint4 q, uint4 x, int s) {
  s = __dp4a(static_cast<int>(q.x), static_cast<int>(x.x), s);
  s = __dp4a(static_cast<int>(q.y), static_cast<int>(x.y), s);
  s = __dp4a(static_cast<int>(q.z), static_cast<int>(x.z), s);
  return __dp4a(static_cast<int>(q.w), static_cast<int>(x.w), s);
}

// N query heads' sums with a page's bounds: L pieces of 16 columns.
template <int L, int N>
__device__ __forceinline__ float heads_bound(const uint4 (*q_pos)[L], const uint4 (*q_neg)[L],
                                             const float* q_step, const uint4* bounds) {
  int s[N];
#pragma unroll
  for (int k = 0; k < N; ++k) s[k] = 0;
#pragma unroll
  for (int c = 0; c < L; ++c) {
    const uint4 lo = bounds[c], hi = bounds[L + c];
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] = dot16(q_neg[k][c], lo, dot16(q_pos[k][c], hi, s[k]));
  }
  float best = -INFINITY;
#pragma unroll
  for (int k = 0; k < N; ++k) best = fmaxf(best, static_cast<float>(s[k]) * q_step[k]);
  return best;
}

// The scores of one (token, kv head)'s pages, 32 neighbouring ones to a warp.
// The warp's pages are copied to shared memory, all under way at once, in rows 16
// bytes longer, so that the lanes' pieces lie in different banks; then each lane
// sums up its own page's: the query heads' pieces are the same for all lanes,
// and no sum crosses them.  (128 of 2,048 to 4,096 pages for 16 tokens, under a
// profiler: with d / 16 lanes to a page and exchanges between them 29 us and 15.3
// million warp instructions, with a bulk copy per page, issued lane by lane, 27 us
// and 12.8 million, as it is 25 us and 11.6 million.)
template <int D>
__global__ void __launch_bounds__(32 * kScoreWarps)
    kv_score_kernel(const SelectArgs a, int chunks) {
  constexpr int L = D / 16;  // 16-byte pieces of a row
  __shared__ __align__(16) uint4 pages_s[kScoreWarps][32][2 * L + 1];
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
  const int b0 = chunk * kScoreWarps * 32;
  // without a choice to make, or pages of this stretch, there is nothing to score
  if (w.state < 1 || newest < a.n_select || b0 >= newest) return;
  const int c = b0 + warp * 32 + lane;
  int page = -1;
  if (c < newest) page = __ldg(pg.table + static_cast<int64_t>(w.b) * pg.cols + c);
  const bool good = page >= 0 && page < pg.num_pages;
  const int64_t at = static_cast<int64_t>(good ? page : 0) * pg.kv_heads + g;
  // a page behind the last, or a bad one, is not sent for: nothing comes of what
  // lies in its place
  const unsigned sent = __ballot_sync(0xffffffffu, good);
#pragma unroll
  for (int i = 0; i < 2 * L; ++i) {
    const int k = i * 32 + lane, slot = k / (2 * L), piece = k % (2 * L);
    const int64_t from = __shfl_sync(0xffffffffu, at, slot);
    if (sent >> slot & 1u)
      copy16_async(smem_u32(&pages_s[warp][slot][piece]), a.bounds + from * 2 * D + piece * 16);
  }
  float scale = 0.f;
  if (good) scale = __ldg(a.bound_scale + at);
  float best = -INFINITY;
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
    if (h0 == 0) {
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
    }
    const uint4* mine = pages_s[warp][lane];
    int h = 0;
    for (; h + 4 <= heads; h += 4)
      best = fmaxf(best, heads_bound<L, 4>(q_pos + h, q_neg + h, q_step + h, mine));
    if (h + 2 <= heads) {
      best = fmaxf(best, heads_bound<L, 2>(q_pos + h, q_neg + h, q_step + h, mine));
      h += 2;
    }
    if (h < heads) best = fmaxf(best, heads_bound<L, 1>(q_pos + h, q_neg + h, q_step + h, mine));
  }
  // + 0: a product that underflows has no sign
  if (c < newest)
    a.scores[(static_cast<int64_t>(t) * pg.kv_heads + g) * pg.cols + c] =
        good ? best * scale + 0.f : __uint_as_float(kBadScore);
}

// --------------------------------------------------------------------- choice

constexpr int kPickKeys = 8192;  // that stay in shared memory; those behind are read again
constexpr int kStaged = 2048;    // places whose pages are looked up together at the end
constexpr int kClose = 512;      // scores of one bin that are compared with one another

// fp32 in the order of unsigned whole numbers; a NaN (an infinity times a scale of
// 0) below all others.
__device__ __forceinline__ unsigned rank_key(float x) {
  const unsigned u = __float_as_uint(x);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The number that a key stands for (a NaN's is one).
__device__ __forceinline__ float score_of(unsigned key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// One block per (token, kv head): the n_select - 1 largest scores, then the
// pages in order.  The smallest of them is looked for among evenly spaced bins
// of the scores' range; the few scores of its bin are compared with one another.
// Should they be many (equal scores, or one far from the rest), they are searched
// by their bits, eight at a time.
template <int kThreads>
__global__ void __launch_bounds__(kThreads) kv_pick_kernel(const SelectArgs a) {
  constexpr int kWarps = kThreads / 32;
  __shared__ unsigned keys[kPickKeys];
  __shared__ int bins[kThreads];
  __shared__ int staged[kStaged];
  __shared__ unsigned close[kClose];
  __shared__ int counts[2][kWarps];
  __shared__ unsigned least[kWarps], most[kWarps];
  __shared__ int found[3];
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
  bins[threadIdx.x] = 0;
  if (threadIdx.x == 0) found[2] = 0;
  // no token need resolve to a sequence whose offsets descend: the first block
  // looks at all of them, while the scores are computed
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < pg.B; b += kThreads)
      if (bad_sequence(pg, a.T, __ldg(a.q_offsets + b), __ldg(a.q_offsets + b + 1),
                       __ldg(pg.kv_len + b)))
        atomicOr(a.err, kErrPages);
  }
  pdl_wait();
  if (w.state == 1 && newest < a.n_select) {
    // every page there is
    bool wrong = false;
    for (int c = threadIdx.x; c <= newest; c += kThreads) {
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
    constexpr int kAtOnce = 8;
    for (int c0 = threadIdx.x; c0 < newest; c0 += kAtOnce * kThreads) {
      float x[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        x[k] = c0 + k * kThreads < newest ? scores[c0 + k * kThreads] : 0.f;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int c = c0 + k * kThreads;
        if (c >= newest) break;
        const unsigned key = rank_key(x[k]);
        wrong = wrong || __float_as_uint(x[k]) == kBadScore;
        if (c < kPickKeys) keys[c] = key;
        lo = min(lo, key);
        hi = max(hi, key);
      }
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
    for (int i = 0; i < kWarps; ++i) {
      lo = min(lo, least[i]);
      hi = max(hi, most[i]);
    }
    // the want-th largest key, and how many of the equal ones are in
    unsigned prefix = hi;
    int left = want;
    if (lo != hi && want > 0) {
      // bins that grow with the score, whatever the rounding; a NaN's, or one of
      // an infinite range, is the first
      const float base = score_of(lo);
      const float per = (kThreads - 1) / (score_of(hi) - base);
      auto bin_of = [&](unsigned key) {
        return min(max(__float2int_rd((score_of(key) - base) * per), 0), kThreads - 1);
      };
      for (int c = threadIdx.x; c < newest; c += kThreads) atomicAdd(&bins[bin_of(key_of(c))], 1);
      __syncthreads();
      // thread i: the scores in bin kThreads - 1 - i and those above
      const int mine = bins[kThreads - 1 - threadIdx.x];
      int incl = mine;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, s);
        if (lane >= s) incl += up;
      }
      if (lane == 31) counts[0][warp] = incl;
      __syncthreads();
      for (int i = 0; i < warp; ++i) incl += counts[0][i];
      if (incl >= left && incl - mine < left) {
        found[0] = kThreads - 1 - threadIdx.x;
        found[1] = left - (incl - mine);
      }
      __syncthreads();
      const int bin = found[0];
      left = found[1];
      for (int c = threadIdx.x; c < newest; c += kThreads) {
        const unsigned key = key_of(c);
        if (bin_of(key) != bin) continue;
        const int i = atomicAdd(&found[2], 1);
        if (i < kClose) close[i] = key;
      }
      bins[threadIdx.x] = 0;
      __syncthreads();
      const int n = found[2];
      if (n <= kClose) {
        for (int i = threadIdx.x; i < n; i += kThreads) {
          const unsigned key = close[i];
          int above = 0, equal = 0;
          for (int k = 0; k < n; ++k) {
            above += close[k] > key ? 1 : 0;
            equal += close[k] == key ? 1 : 0;
          }
          if (above < left && above + equal >= left) {  // equal ones agree
            found[0] = static_cast<int>(key);
            found[1] = left - above;
          }
        }
        __syncthreads();
        prefix = static_cast<unsigned>(found[0]);
        left = found[1];
      } else {
        prefix = 0u;
        for (int shift = 24; shift >= 0; shift -= 8) {
          for (int c = threadIdx.x; c < newest; c += kThreads) {
            const unsigned key = key_of(c);
            if (bin_of(key) == bin && (shift == 24 || key >> (shift + 8) == prefix >> (shift + 8)))
              atomicAdd(&bins[(key >> shift) & 255u], 1);
          }
          __syncthreads();
          if (warp == 0) {
            // lane l: bins 255 - 8 l and the seven below
            int part[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              sum += part[i] = bins[255 - 8 * lane - i];
              bins[255 - 8 * lane - i] = 0;
            }
            int upto = sum;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
              const int up = __shfl_up_sync(0xffffffffu, upto, s);
              if (lane >= s) upto += up;
            }
            int before = upto - sum;
            if (before < left && upto >= left) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                if (before < left && before + part[i] >= left) {
                  found[0] = 255 - 8 * lane - i;
                  found[1] = left - before;
                }
                before += part[i];
              }
            }
          }
          __syncthreads();
          prefix |= static_cast<unsigned>(found[0]) << shift;
          left = found[1];
          __syncthreads();
        }
      }
    }
    // a warp takes a stretch of neighbouring columns: first its number of
    // larger and of equal keys, then the places
    const int stretch = (newest + kThreads - 1) / kThreads * 32;
    const int s0 = warp * stretch, s1 = min(newest, s0 + stretch);
    int above = 0, equal = 0;
#pragma unroll 4
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
      if (is_above || (is_equal && ne < left)) {
        const int place = na + min(ne, left);
        if (place < kStaged)
          staged[place] = c;
        else
          out[place] = __ldg(row + c);
      }
      a0 += __popc(ma);
      e0 += __popc(me);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < min(want, kStaged); i += kThreads)
      out[i] = __ldg(row + staged[i]);
    if (threadIdx.x == 0) out[want] = __ldg(row + newest);
    picked = a.n_select;
  }
  if (bad) {
    if (threadIdx.x == 0) atomicOr(a.err, kErrPages);
    __syncthreads();
    picked = 0;
  }
  for (int i = picked + threadIdx.x; i < a.n_select; i += kThreads) out[i] = -1;
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
  if (units > 0x7fffffffLL) return MHA_ERR_UNSUPPORTED;
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
  const int chunks = (pages->table_cols + kScoreWarps * 32 - 1) / (kScoreWarps * 32);
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
  // a thread for every two or three scores (1,024 of them: a batch over 2 to 4 K
  // pages 30 us instead of 36, one conversation over 2 K pages 9.0 instead of 8.6)
  const bool many = pages->table_cols > 2560;
  cfg.blockDim = dim3(many ? 1024 : 512);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, many ? kv_pick_kernel<1024> : kv_pick_kernel<512>, a) != cudaSuccess)
    return MHA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MHA_OK : MHA_ERR_CUDA;
}

}  // extern "C"
