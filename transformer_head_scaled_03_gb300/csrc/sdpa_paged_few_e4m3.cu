// sdpa_paged_few_e4m3.cu -- paged attention of few query rows over a cache in 8
// bits: at most 16 rows (new tokens x query heads per key/value head) per
// sequence and key/value head.
//
// The shape is that of sdpa_paged_few.cu (keys are the products' M side, a CTA
// is one split of one (sequence, kv head), clusters merge the splits), with
// the codes as they lie in the pages for operands:
//   S^T = K_codes Q^T      tcgen05 kind::f8f6f4, M = 128 keys, K = d
//   softmax over keys      warps 0-3, one key (TMEM lane) per thread
//   O^T = V_codes^T W^T    M = d, K = 128 keys
// so no byte of the cache is converted.  What is not 8 bits wide is taken as
// two e4m3 parts (ptx_e4m3.cuh), which lie side by side on the products' N
// side, 2 U columns for U query slots: a row of Q over a power of two that
// brings its largest element to 224..448, and the weights.  A page's key scale
// multiplies its scores, a thread's own; its value scale v joins the score, over
// one value scale c of the CTA, so that a weight's parts are held against the
// largest product of weight and value scale of its own row:
//   t_j = q . codes_j * kscale_j + log2(v_j / c),   m = max t
//   w_j = 256 * 2^(t_j - m),  l = sum w_j c / v_j,  o = c * sum_j w_j codes_j / l
// A key whose value scale is 0 meets no values (its w is 0): it is in l, and in m as if
// its scale were 2^-30 c, which keeps l in range.
//
// Half the bytes of the bf16 form for the same tiles: bound by HBM up to eight
// rows, by the softmax's chain with more.  Measured: 16 sequences of 16 to 32 K
// tokens, 32 heads on 8 kv heads, d = 128: 118 us, 6.8 TB/s of cache (the bf16
// cache: 215 us); 64 heads on 8 121 us, 128 on 8 144 us (190 with the slots'
// scales and last keys in registers, which spilled); d = 64 78 us; 64 sequences
// of 200 to 1000 tokens 26 us; one token over 700 keys 7.5 us on the device.
// Keys of scale 0 let m down by 60 instead of 30 and l carried in two steps, which
// would allow for value scales 2^100 apart beside zeros, too, took 154 us with 128
// heads.
#include <math.h>
#include <stdint.h>

#include <cuda_bf16.h>

#include "ptx_e4m3.cuh"
#include "sdpa_paged.cuh"

namespace mha {
namespace {

constexpr int kKeys = 128;             // keys per tile
constexpr int kSlots = kPagedFewRows;  // query rows at most
constexpr int kThreads = 192;          // warps 0-3 softmax, 4 TMA, 5 MMA
constexpr int kTmaWarp = 4;
constexpr int kMmaWarp = 5;
constexpr int kMaxSortedBatch = 256;
constexpr float kQUp = 16.f;   // what the second parts of Q (at most 16 of 448) are times
constexpr float kWUp = 32.f;   // and of the weights (at most 8 of 256)
constexpr float kWTop = 256.f;

// U: query slots that the softmax works on; kAlone: a CTA per SM at most.
template <int D, int U, bool kAlone>
struct Few8Cfg {
  static_assert(D == 64 || D == 128, "head dim");
  static_assert(U == 4 || U == 8 || U == 16, "slots");
  static constexpr int N = 2 * U < 16 ? 16 : 2 * U;  // the products' columns
  static constexpr uint32_t kTmemCols = N == 16 ? 64u : 128u;  // S^T x 2, O^T x 2
  // Two CTAs share an SM, or three with few slots at d = 64, where a tile is half
  // the bytes for the same softmax (16 sequences of 16 to 32 K keys, 32 heads on
  // 8: 83 -> 76 us; at d = 128 three took 121 us instead of 117).
  static constexpr int kCtas = kAlone ? 1 : D == 64 && U == 4 ? 3 : 2;
  static constexpr int NR = D == 128 ? (kAlone ? 12 : 6) : kAlone ? 22 : kCtas == 3 ? 7 : 11;
  static constexpr int kTile = kKeys * D;
  static constexpr int kPBuf = N * 128;  // W^T of one tile: N rows x 128 keys
  static constexpr int kOffRing = 0;
  static constexpr int kOffQ = kOffRing + NR * kTile;  // N rows x d
  static constexpr int kOffP = kOffQ + N * 128;
  static constexpr int kOffRed = kOffP + 2 * kPBuf;  // [3][4 warps][16 + 4] f32
  static constexpr int kRedRow = kSlots + 4;         // the slots' maxima, the scales'
  static constexpr int kOffX = kOffRing;
  static_assert(few_merge_bytes(D) <= kTile, "the merge fits a slot");
  static constexpr int kOffBar = kOffRed + 3 * 4 * kRedRow * 4;
  static constexpr int bQ = 0;
  __host__ __device__ static constexpr int bF(int s) { return 1 + s; }
  __host__ __device__ static constexpr int bE(int s) { return 1 + NR + s; }
  __host__ __device__ static constexpr int bS(int i) { return 1 + 2 * NR + i; }
  __host__ __device__ static constexpr int bP(int i) { return bS(0) + 2 + i; }
  __host__ __device__ static constexpr int bO(int i) { return bS(0) + 4 + i; }
  __host__ __device__ static constexpr int bRed(int i) { return bS(0) + 6 + i; }
  static constexpr int bDrain = 1 + 2 * NR + 8;
  static constexpr int kNumBars = bDrain + 1;
  static constexpr int kOffMisc = kOffBar + 8 * kNumBars;
  // of every slot, [16]: its row's scale times the softmax's, its last key
  static constexpr int kOffQs = (kOffMisc + 16 + 15) / 16 * 16;
  static constexpr int kOffLast = kOffQs + kSlots * 4;
  // lengths and offsets of the sequences, while they are ranked
  static constexpr int kOffSeq = kOffLast + kSlots * 4;
  static constexpr int kSeqBytes = (2 * kMaxSortedBatch + 2) * 4;
  // the M = 128 operand of a d = 64 product reads the 8 KB after a V tile as
  // its unused upper half: there is that much after the last slot
  static constexpr int kEnd =
      kOffSeq + kSeqBytes > kOffQ + kTile ? kOffSeq + kSeqBytes : kOffQ + kTile;
  static constexpr int kSmemBytes = kEnd + 1024;  // + alignment slack
  static_assert(kOffQ % 1024 == 0 && kOffP % 1024 == 0, "swizzle atoms");
  static_assert(kSmemBytes + 1024 <= 228 * 1024 / kCtas, "CTAs per SM");
};

// Places of K(j) and V(j) in the ring's order, for T tiles.
__device__ __forceinline__ int place_of_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int place_of_v(int j, int T) { return j + 1 < T ? 2 * j + 2 : 2 * j + 1; }

// N columns of this thread's lane in tensor memory (8, 16 or 32).
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 8) {
    tmem_ld8_sync(taddr, r);
  } else if constexpr (N == 16) {
    tmem_ld16_sync(taddr, r);
  } else {
    static_assert(N == 32, "columns");
    tmem_ld32(taddr, r);
    tmem_ld_wait(r);
  }
}

template <int D, int U, bool kAlone>
__global__ void __launch_bounds__(kThreads, Few8Cfg<D, U, kAlone>::kCtas)
    sdpa_paged_few_e4m3_kernel(const __nv_bfloat16* __restrict__ Q, int64_t q_stride,
                               const __grid_constant__ CUtensorMap tmK,
                               const __grid_constant__ CUtensorMap tmV, const PagedParams p) {
  using C = Few8Cfg<D, U, kAlone>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + C::kOffMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::kOffMisc + 4);
  volatile int* bad_page = reinterpret_cast<volatile int*>(gbase + C::kOffMisc + 8);
  auto bar = [base](int i) -> uint32_t { return base + C::kOffBar + 8u * i; };

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const WaitCtl ctl{abort_flag, p.err, p.limit_ns};

  if (threadIdx.x == 0) {
    mbar_init(bar(C::bQ), 128);
    for (int s = 0; s < C::NR; ++s) {
      mbar_init(bar(C::bF(s)), 1);
      mbar_init(bar(C::bE(s)), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::bS(i)), 1);
      mbar_init(bar(C::bP(i)), 128);
      mbar_init(bar(C::bO(i)), 1);
      mbar_init(bar(C::bRed(i)), 128);
    }
    mbar_init(bar(C::bDrain), 1);
    *abort_flag = 0;
    *bad_page = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc<C::kTmemCols>(smem_u32(tmem_slot));
    tmem_relinquish();
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  float* red = reinterpret_cast<float*>(gbase + C::kOffRed);
  float* q_scale = reinterpret_cast<float*>(gbase + C::kOffQs);
  int* last_key = reinterpret_cast<int*>(gbase + C::kOffLast);
  float* xm = reinterpret_cast<float*>(gbase + C::kOffX);
  float* xl = xm + kSlots;
  float* xo = xl + kSlots;

  // ---- this CTA's (sequence, kv head) and key tiles, longest sequences first
  // (see sdpa_paged_few.cu)
  const int split = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.splits));
  const int slot = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.splits));
  const int g = slot % p.kv_heads;
  int b = slot / p.kv_heads;
  const bool sorted = p.B > 1 && p.B <= kMaxSortedBatch;
  int* lens_s = reinterpret_cast<int*>(gbase + C::kOffSeq);
  int* off_s = lens_s + kMaxSortedBatch;
  int* pick = off_s + kMaxSortedBatch + 1;
  PagedSeq seq{};
  if (sorted) {
    for (int i = threadIdx.x; i <= p.B; i += kThreads) {
      off_s[i] = paged_offset(p, i);
      if (i < p.B) lens_s[i] = __ldg(p.kv_len + i);
    }
  } else {
    seq = paged_seq(p, b);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  if (sorted) {
    const int want = b;
    for (int c = threadIdx.x; c < p.B; c += kThreads) {
      const int lc = lens_s[c];
      int rank = 0;
#pragma unroll 8
      for (int o = 0; o < p.B; ++o) {
        const int lo = lens_s[o];
        rank += (lo > lc || (lo == lc && o < c)) ? 1 : 0;
      }
      if (rank == want) *pick = c;
    }
    __syncthreads();
    b = *pick;
    seq = paged_seq_of(p, off_s[b], off_s[b + 1], lens_s[b]);
  }
  const int rows = seq.n * p.G;  // query slots in use: slot = token * G + head of the group
  const int len = seq.len;
  const int n_tiles = seq.bad_len || rows == 0 ? 0 : (len + kKeys - 1) / kKeys;
  const int t_begin = static_cast<int>(static_cast<long long>(n_tiles) * split / p.splits);
  const int t_end = static_cast<int>(static_cast<long long>(n_tiles) * (split + 1) / p.splits);
  const int T = t_end - t_begin;
  if ((seq.bad_len || seq.bad_offsets) && split == 0 && threadIdx.x == 0)
    atomicOr(p.err, kErrPages);

  if (warp == kTmaWarp) {
    // ------------------------------------------------------------ producer
    if (T > 0) {
      using Boxes = PageBoxes<kKeys, 1, D>;
      const int32_t* row = table_row(p, b, g);
      Boxes cur, nxt;
      cur.fetch(p, row, t_begin * kKeys, len, lane);
      int issued = 0;
      // the box of every lane into the ring's next slot; false: gave up
      auto load = [&](const Boxes& boxes, const CUtensorMap* map, int key0) {
        const int s = issued % C::NR;
        const uint32_t bytes = boxes.bytes(p);
        if (!mbar_wait_warp(bar(C::bE(s)), ((issued / C::NR) & 1) ^ 1u, ctl)) return false;
        if (lane == 0) mbar_expect_tx(bar(C::bF(s)), bytes);
        __syncwarp();
        boxes.load(p, map, base + C::kOffRing + s * C::kTile, bar(C::bF(s)), key0, g, lane);
        ++issued;
        return true;
      };
      const int first = t_begin * kKeys;
      bool ok = load(cur, &tmK, first);
      for (int j = 0; ok && j < T; ++j) {
        if (cur.bad(p)) {
          *bad_page = 1;
          atomicOr(p.err, kErrPages);
        }
        // the next tile's keys go before this tile's values
        const int key0 = first + j * kKeys;
        if (j + 1 < T) {
          nxt.fetch(p, row, key0 + kKeys, len, lane);
          if (!(ok = load(nxt, &tmK, key0 + kKeys))) break;
        }
        ok = load(cur, &tmV, key0);
        cur = nxt;
      }
      // let every issued copy land before the CTA can exit
      if (lane == 0) {
        for (int x = max(0, issued - C::NR); x < issued; ++x)
          paged_wait_drain(bar(C::bF(x % C::NR)), (x / C::NR) & 1, p.limit_ns);
      }
    }
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------- MMA issuer
    // Order: S(0), S(1), then per tile j: O(j) once W(j) is published, and
    // S(j+2) into the S buffer that W(j)'s publication has just released.
    if (lane == 0 && T > 0) {
      constexpr uint32_t kIdS = idesc_e4m3_f32(kKeys, C::N, false, false);
      constexpr uint32_t kIdO = idesc_e4m3_f32(128, C::N, true, false);
      const uint64_t q_desc = sdesc_rows<D>(base + C::kOffQ, 16, 8 * D);
      const uint64_t k_desc = sdesc_rows<D>(base + C::kOffRing, 16, 8 * D);
      const uint64_t v_desc = sdesc_rows<D>(base + C::kOffRing, C::kTile, 8 * D);
      const uint64_t p_desc = sdesc_rows<128>(base + C::kOffP, 16, 1024);
      auto issue_s = [&](int st, int buf) {
        const uint64_t kd = k_desc + static_cast<uint64_t>((st * C::kTile) >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks)
          umma_f8_ss(tmem + buf * C::N, kd + 2 * ks, q_desc + 2 * ks, kIdS, ks > 0 ? 1u : 0u);
      };
      auto issue_o = [&](int st, int buf) {
        const uint64_t vd = v_desc + static_cast<uint64_t>((st * C::kTile) >> 4);
        const uint64_t pd = p_desc + static_cast<uint64_t>((buf * C::kPBuf) >> 4);
#pragma unroll
        for (int ks = 0; ks < kKeys / 32; ++ks)
          umma_f8_ss(tmem + (2 + buf) * C::N, vd + static_cast<uint64_t>((ks * 32 * D) >> 4),
                     pd + 2 * ks, kIdO, ks > 0 ? 1u : 0u);
      };
      auto wait_full = [&](int x) {
        return mbar_wait(bar(C::bF(x % C::NR)), (x / C::NR) & 1, ctl);
      };
      bool ok = mbar_wait(bar(C::bQ), 0, ctl);
      for (int j = 0; ok && j < 2 && j < T; ++j) {
        const int x = place_of_k(j);
        if (!(ok = wait_full(x))) break;
        tc_fence_after();
        issue_s(x % C::NR, j);
        umma_commit(bar(C::bS(j)));
        umma_commit(bar(C::bE(x % C::NR)));
      }
      for (int j = 0; ok && j < T; ++j) {
        const int x = place_of_v(j, T);
        const int buf = j & 1;
        if (!(ok = mbar_wait(bar(C::bP(buf)), (j >> 1) & 1, ctl))) break;
        if (!(ok = wait_full(x))) break;
        tc_fence_after();
        issue_o(x % C::NR, buf);
        umma_commit(bar(C::bO(buf)));
        umma_commit(bar(C::bE(x % C::NR)));
        if (j + 2 < T) {
          const int y = place_of_k(j + 2);
          if (!(ok = wait_full(y))) break;
          tc_fence_after();
          issue_s(y % C::NR, buf);
          umma_commit(bar(C::bS(buf)));
          umma_commit(bar(C::bE(y % C::NR)));
        }
      }
      // every issued MMA completes before tensor memory is released
      umma_commit(bar(C::bDrain));
      paged_wait_drain(bar(C::bDrain), 0, p.limit_ns);
    }
  } else {
    // ------------------------------------------------------------- softmax
    // Thread r owns key r of every S^T tile and row r (output column r) of
    // every O^T tile.
    const int r = warp * 32 + lane;
    const uint32_t lane_bits = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tS = tmem + lane_bits;
    const uint32_t tO = tmem + lane_bits + 2 * C::N;
    const bool o_rows = warp * 32 < D;  // warp-uniform

    // this thread's key of the next tiles: its page two tiles ahead, its scales
    // one ahead, so that neither look-up is waited for
    const int32_t* row = T > 0 ? table_row(p, b, g) : nullptr;
    auto page_of = [&](int j) {
      const int key = (t_begin + j) * kKeys + r;
      return j < T && key < len ? __ldg(row + (key >> p.page_shift)) : -1;
    };
    auto scales_of = [&](int page, float& sk, float& sv) {
      const bool good = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages);
      const int64_t at = static_cast<int64_t>(page) * p.kv_heads + g;
      sk = good ? __ldg(p.k_scale + at) : 0.f;
      sv = good ? __ldg(p.v_scale + at) : 0.f;
    };
    int page = page_of(0), page1 = page_of(1);
    // c: the largest value scale of the first tile that has one above 0, from the
    // warps' largest, which are handed over with other things
    float c = 0.f;
    auto largest_of_warps = [](const float* at) {
      at += kSlots;
      return fmaxf(fmax3(at[0], at[C::kRedRow], at[2 * C::kRedRow]), at[3 * C::kRedRow]);
    };
    float* lsum = red + 2 * 4 * C::kRedRow;
    float sk, sv;
    scales_of(page, sk, sv);

    if (T > 0) {
      // Q as two parts: eight threads to a row, D / 8 columns each
      const int qr = r >> 3, part = r & 7;
      constexpr int n = D / 8;
      float x[n];
      const int i = div_by_group(p, qr);
      const bool here = qr < rows;
      const uint4* from = reinterpret_cast<const uint4*>(
          Q + (seq.q0 + i) * q_stride + static_cast<int64_t>(g * p.G + qr - i * p.G) * D + part * n);
      float top = 0.f;
#pragma unroll
      for (int v = 0; v < n / 8; ++v) {
        const uint4 u = here ? __ldg(from + v) : make_uint4(0u, 0u, 0u, 0u);
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = __bfloat1622float2(h[k]);
          x[8 * v + 2 * k] = f.x;
          x[8 * v + 2 * k + 1] = f.y;
        }
      }
#pragma unroll
      for (int k = 0; k < n; ++k) {
        if (fabsf(x[k]) < INFINITY)
          top = fmaxf(top, fabsf(x[k]));
        else
          x[k] = NAN;  // the row's scores, as infinities would make them in the end
      }
#pragma unroll
      for (int s = 1; s < 8; s <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
      float inv;
      const float scale = part_scale_of(top, &inv);
      if (part == 0) {
        q_scale[qr] = scale * p.scale_log2;
        last_key[qr] = qr >= rows ? -1 : p.causal ? len - seq.n + i : len - 1;
      }
      if (qr < U) {
        uint32_t hi[n / 4], lo[n / 4];
#pragma unroll
        for (int k = 0; k < n / 4; ++k) {
          uint32_t a0, a1, b0, b1;
          two_parts(x[4 * k] * inv, x[4 * k + 1] * inv, kQUp, &a0, &b0);
          two_parts(x[4 * k + 2] * inv, x[4 * k + 3] * inv, kQUp, &a1, &b1);
          hi[k] = a0 | a1 << 16;
          lo[k] = b0 | b1 << 16;
        }
        uint8_t* q0 = gbase + C::kOffQ;
        if constexpr (D == 128) {
          *reinterpret_cast<uint4*>(q0 + piece_at<D>(qr, part)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(q0 + piece_at<D>(qr + U, part)) =
              make_uint4(lo[0], lo[1], lo[2], lo[3]);
        } else {
          *reinterpret_cast<uint2*>(q0 + piece_at<D>(qr, part / 2) + (part & 1) * 8) =
              make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(q0 + piece_at<D>(qr + U, part / 2) + (part & 1) * 8) =
              make_uint2(lo[0], lo[1]);
        }
      }
      if constexpr (2 * U < C::N) {
        // the products' columns behind both parts: zeros, of Q and of the weights
        for (int v = r; v < (C::N - 2 * U) * D / 16; v += 128)
          *reinterpret_cast<uint4*>(gbase + C::kOffQ + 2 * U * D + v * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        for (int v = r; v < (C::N - 2 * U) * 8 * 2; v += 128)
          *reinterpret_cast<uint4*>(gbase + C::kOffP + (v & 1) * C::kPBuf + 2 * U * 128 + (v >> 1) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(C::bQ));
      const float wc = warp_max_f32(sv);
      if (lane == 0) lsum[warp * C::kRedRow + kSlots] = wc;
      softmax_bar();  // the rows' scales are there
      c = largest_of_warps(lsum);
    }

    float m[U], l[U], acc[U], alpha_prev[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      m[q] = -INFINITY;
      l[q] = 0.f;
      acc[q] = 0.f;
      alpha_prev[q] = 1.f;
    }
    // keys that every slot sees (one not in use may see any: its sums are not
    // stored)
    const int all_see = p.causal ? len - seq.n + 1 : len;
    // W^T store address of key r: 16-byte piece and byte of a 128-byte row
    const int piece = r >> 4;
    uint8_t* p_key = gbase + C::kOffP + (r & 15);
    bool ok = true;
    for (int j = 0; j < T; ++j) {
      const int buf = j & 1;
      const uint32_t par = (j >> 1) & 1;
      const int key = (t_begin + j) * kKeys + r;
      float sk1, sv1;
      scales_of(page1, sk1, sv1);
      page1 = page_of(j + 2);
      float* rb = red + buf * 4 * C::kRedRow;
      // value scales of a sequence, but for zeros, lie within 2^100 of each other
      const bool none = !(sv > 0.f);
      const float ratio = none ? 0x1p-30f : fminf(fmaxf(sv / c, 0x1p-100f), 0x1p100f);
      const float v = __log2f(ratio), iv = ex2_approx(-v);
      const float times = none ? 0.f : kWTop;
      if (!(ok = mbar_wait_warp(bar(C::bS(buf)), par, ctl))) break;
      tc_fence_after();
      float s[U];
      {
        uint32_t sr[2 * U];
        tmem_ld_cols<2 * U>(tS + buf * C::N, sr);
#pragma unroll
        for (int q = 0; q < U; q += 4) {
          const float4 f = *reinterpret_cast<const float4*>(q_scale + q);
          const float qs[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            s[q + k] = fmaf(
                fmaf(__uint_as_float(sr[U + q + k]), 1.f / kQUp, __uint_as_float(sr[q + k])),
                sk * qs[k], v);
        }
        if ((t_begin + j + 1) * kKeys > all_see) {
#pragma unroll
          for (int q = 0; q < U; ++q) s[q] = key <= last_key[q] ? s[q] : -INFINITY;
        }
      }
      {
        float wm[U];
#pragma unroll
        for (int q = 0; q < U; ++q) wm[q] = warp_max_f32(s[q]);
        if (lane == 0) {
          float4* dst = reinterpret_cast<float4*>(rb + warp * C::kRedRow);
#pragma unroll
          for (int i = 0; i < U / 4; ++i)
            dst[i] = make_float4(wm[4 * i], wm[4 * i + 1], wm[4 * i + 2], wm[4 * i + 3]);
        }
        if (c == 0.f) {  // the same for every thread: the next tile's
          const float wc = warp_max_f32(sv1);
          if (lane == 0) rb[warp * C::kRedRow + kSlots] = wc;
        }
      }
      mbar_arrive(bar(C::bRed(buf)));
      if (!(ok = mbar_wait_warp(bar(C::bRed(buf)), par, ctl))) break;
      if (c == 0.f) c = largest_of_warps(rb);
      float alpha[U];
#pragma unroll
      for (int i = 0; i < U / 4; ++i) {
        const float4 a0 = reinterpret_cast<const float4*>(rb)[i];
        const float4 a1 = reinterpret_cast<const float4*>(rb + C::kRedRow)[i];
        const float4 a2 = reinterpret_cast<const float4*>(rb + 2 * C::kRedRow)[i];
        const float4 a3 = reinterpret_cast<const float4*>(rb + 3 * C::kRedRow)[i];
        const float t4[4] = {fmaxf(fmax3(a0.x, a1.x, a2.x), a3.x),
                             fmaxf(fmax3(a0.y, a1.y, a2.y), a3.y),
                             fmaxf(fmax3(a0.z, a1.z, a2.z), a3.z),
                             fmaxf(fmax3(a0.w, a1.w, a2.w), a3.w)};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int q = 4 * i + u;
          const float mn = fmaxf(m[q], t4[u]);
          const float at = mn == -INFINITY ? 0.f : mn;  // a slot with no visible key yet
          alpha[q] = ex2_approx(m[q] - at);
          const float pq = ex2_approx(s[q] - at);
          l[q] = fmaf(pq, iv, l[q] * alpha[q]);
          m[q] = mn;
          s[q] = pq * times;
        }
      }
      // W^T(j): rows q (first parts) and U + q (second), key r, 128-byte swizzle
      uint8_t* pb = p_key + buf * C::kPBuf;
#pragma unroll
      for (int q = 0; q < U; q += 2) {
        uint32_t first, second;
        two_parts(s[q], s[q + 1], kWUp, &first, &second);
        pb[piece_at<128>(q, piece)] = static_cast<uint8_t>(first);
        pb[piece_at<128>(q + 1, piece)] = static_cast<uint8_t>(first >> 8);
        pb[piece_at<128>(U + q, piece)] = static_cast<uint8_t>(second);
        pb[piece_at<128>(U + q + 1, piece)] = static_cast<uint8_t>(second >> 8);
      }
      if ((t_begin + j + 1) * kKeys > len) {
        // V rows behind the length: zero them once the tile has landed (it
        // stays until this tile's product, which waits for the arrive below)
        const int x = place_of_v(j, T);
        if (!(ok = mbar_wait_warp(bar(C::bF(x % C::NR)), (x / C::NR) & 1, ctl))) break;
        if (key >= len) {
          uint8_t* v_row = gbase + C::kOffRing + x % C::NR * C::kTile + r * D;
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            *reinterpret_cast<uint4*>(v_row + i * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(bar(C::bP(buf)));
      if (j > 0) {
        const int pj = j - 1;
        if (!(ok = mbar_wait_warp(bar(C::bO(pj & 1)), (pj >> 1) & 1, ctl))) break;
        tc_fence_after();
        if (o_rows) {
          uint32_t orr[2 * U];
          tmem_ld_cols<2 * U>(tO + (pj & 1) * C::N, orr);
#pragma unroll
          for (int q = 0; q < U; ++q)
            acc[q] = fmaf(acc[q], alpha_prev[q],
                          fmaf(__uint_as_float(orr[U + q]), 1.f / kWUp, __uint_as_float(orr[q])));
        }
      }
#pragma unroll
      for (int q = 0; q < U; ++q) alpha_prev[q] = alpha[q];
      sk = sk1;
      sv = sv1;
    }
    if (ok && T > 0) {
      const int pj = T - 1;
      if ((ok = mbar_wait_warp(bar(C::bO(pj & 1)), (pj >> 1) & 1, ctl))) {
        tc_fence_after();
        if (o_rows) {
          uint32_t orr[2 * U];
          tmem_ld_cols<2 * U>(tO + (pj & 1) * C::N, orr);
#pragma unroll
          for (int q = 0; q < U; ++q)
            acc[q] = fmaf(acc[q], alpha_prev[q],
                          fmaf(__uint_as_float(orr[U + q]), 1.f / kWUp, __uint_as_float(orr[q])));
        }
      }
    }
    tc_fence_before();
    // denominator: sum l over the 128 key lanes
#pragma unroll
    for (int q = 0; q < U; ++q) {
#pragma unroll
      for (int sh = 16; sh > 0; sh >>= 1) l[q] += __shfl_xor_sync(0xffffffffu, l[q], sh);
    }
    if (lane == 0) {
      float4* dst = reinterpret_cast<float4*>(lsum + warp * C::kRedRow);
#pragma unroll
      for (int i = 0; i < U / 4; ++i)
        dst[i] = make_float4(l[4 * i], l[4 * i + 1], l[4 * i + 2], l[4 * i + 3]);
    }
    softmax_bar();
    const bool failed = *abort_flag != 0;
    if (failed) *bad_page = 1;  // a failed split spoils the rows
    auto sum_of = [&](int q) {
      return lsum[q] + lsum[C::kRedRow + q] + lsum[2 * C::kRedRow + q] + lsum[3 * C::kRedRow + q];
    };
    // a split's outputs are merged as they would be alone, with the logarithm of its
    // sum: the maxima of splits, which hold value scales, may lie further apart than
    // fp32 reaches
    if (threadIdx.x < kSlots) {
      const int q = threadIdx.x;
      float mq = -INFINITY;
#pragma unroll
      for (int k = 0; k < U; ++k) mq = k == q ? m[k] : mq;
      const float sum = failed || q >= U ? 0.f : sum_of(q);
      xm[q] = sum != 0.f ? mq + __log2f(sum) : -INFINITY;  // NaN stays NaN
      xl[q] = sum != 0.f ? 1.f : 0.f;
    }
    if (o_rows && r < D) {
      const float back = c * (1.f / kWTop);
#pragma unroll
      for (int q = 0; q < U; ++q) {
        const float sum = sum_of(q);
        xo[q * D + r] = sum != 0.f ? acc[q] * (back / sum) : 0.f;
      }
    }
  }

  __syncwarp();
  cluster_sync();  // every split's m, l, O and bad-page flag are in its shared memory
  if (warp < 4) few_merge<D>(p, seq, g, split, xm, bad_page);
  __syncwarp();
  cluster_sync();  // no CTA leaves while another still reads its shared memory
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc<C::kTmemCols>(tmem);
  }
}

template <int D, int U, bool kAlone>
cudaError_t launch_as(const PagedSdpaArgs& a, const DeviceCtl& ctl) {
  using C = Few8Cfg<D, U, kAlone>;
  CUtensorMap k, v;
  if (!paged_tensor_maps_e4m3(a, D, kKeys, &k, &v)) return cudaErrorInvalidValue;
  const int64_t clusters = static_cast<int64_t>(a.pages.B) * a.pages.kv_heads;
  if (clusters * a.splits > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  auto kern = sdpa_paged_few_e4m3_kernel<D, U, kAlone>;
  static std::atomic<uint64_t> attributes_set{0};
  cudaError_t e = paged_kernel_attributes(reinterpret_cast<const void*>(kern), C::kSmemBytes,
                                          &attributes_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * a.splits));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(a.splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, static_cast<const __nv_bfloat16*>(a.Q), a.q_stride, k, v,
                         paged_params(a, ctl));
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D, int U>
cudaError_t launch_slots(PagedSdpaArgs a, const DeviceCtl& ctl) {
  const int64_t clusters = static_cast<int64_t>(a.pages.B) * a.pages.kv_heads;
  if (a.splits == 0)
    a.splits = paged_default_splits(
        clusters, static_cast<int64_t>(a.pages.cols) << a.pages.page_shift, kThreads,
        Few8Cfg<D, U, false>::kSmemBytes, true);
  const bool alone =
      clusters <= paged_resident_clusters(kThreads, Few8Cfg<D, U, true>::kSmemBytes, a.splits);
  return alone ? launch_as<D, U, true>(a, ctl) : launch_as<D, U, false>(a, ctl);
}

template <int D>
cudaError_t launch_impl(const PagedSdpaArgs& a, const DeviceCtl& ctl) {
  const int64_t rows = static_cast<int64_t>(a.max_new) * a.G;
  return rows <= 4 ? launch_slots<D, 4>(a, ctl)
                   : rows <= 8 ? launch_slots<D, 8>(a, ctl) : launch_slots<D, 16>(a, ctl);
}

}  // namespace

cudaError_t launch_sdpa_paged_few_e4m3(const PagedSdpaArgs& a, const DeviceCtl& ctl) {
  return a.pages.d == 64 ? launch_impl<64>(a, ctl) : launch_impl<128>(a, ctl);
}

}  // namespace mha
