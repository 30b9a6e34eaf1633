// sdpa_paged_few.cu -- paged attention of few query rows: at most 16 rows
// (new tokens x query heads per key/value head) per sequence and key/value
// head, the decoding of one or a few tokens.
//
// One CTA = one split of one (sequence, kv head): tiles of 128 keys, each
// gathered from its pages by TMA boxes of a page's rows, one lane of the
// producer warp per box.
//   S^T = K_tile Q^T      tcgen05, M = 128 keys, N = 16 query slots, K = d
//   softmax over keys     warps 0-3, one key (TMEM lane) per thread
//   O^T = V_tile^T P^T    tcgen05, M = d, N = 16, K = 128 keys
//   merge (cluster)       o = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s
// Keys are the M side because 16 query rows would fill an eighth of it.  The
// query heads that share a key/value head are query slots of one CTA, so
// every page is read once.  The rows of the last page behind the sequence's
// length hold anything, NaN too: their scores are replaced and their V rows
// zeroed in shared memory before the product, where 0 * NaN would reach the
// sums.
//
// At 16 slots a byte of the cache meets at most 16 flops: bound by HBM, so
// the pipeline is sized for bytes in flight (two CTAs of 96 KB per SM).
// Measured: 16 sequences of 16 to 32 K tokens, 32 heads on 8 kv heads, d = 128:
// 218 us, 7.1 TB/s of cache (DRAM at 89 % of its nominal rate); 64 sequences of
// 200 to 1000 tokens: 45 us, where a CTA lives for five tiles and its start
// and merge count (one CTA per SM with 64 KB stages: 70 us); one token over
// 700 keys: 8 us on the device.
#include <math.h>
#include <stdint.h>

#include <cuda_bf16.h>

#include "sdpa_paged.cuh"

namespace mha {
namespace {

constexpr int kKeys = 128;      // keys per tile: MMA M of S^T, MMA K of O^T
constexpr int kSlots = kPagedFewRows;  // MMA N of both products
constexpr int kSub = 16384;     // one 128-row x 64-column bf16 block
constexpr int kQBox = 2048;     // 16 rows x 64 columns
constexpr int kPBuf = 4096;     // P^T of one tile: 16 rows x 128 keys bf16
constexpr int kThreads = 192;   // warps 0-3 softmax, 4 TMA, 5 MMA
constexpr int kTmaWarp = 4;
constexpr int kMmaWarp = 5;
constexpr uint32_t kTmemCols = 64;  // S^T x 2 (cols 0-31), O^T x 2 (cols 32-63)
constexpr int kMaxSortedBatch = 256;

// kAlone: the launch has a CTA per SM at most.
template <int D, bool kAlone>
struct FewCfg {
  static_assert(D == 64 || D == 128, "head dim");
  static constexpr int KB = D / 64;
  // K and V tiles go through one ring in the order in which the products take
  // them (K0 K1 V0 K2 V1 K3 ...), so that its slots, 32 KB at d = 128 and 16 KB
  // at d = 64, are all under way or in use.  Two CTAs share an SM, with three
  // slots (five) each: one's set-up, first loads and merge run under the
  // other's stream.  A CTA alone on its SM takes six (eleven): 64 CTAs of 32
  // tiles 51 -> 46 us, 128 of 16 about the same.
  static constexpr int NR = D == 128 ? (kAlone ? 6 : 3) : kAlone ? 11 : 5;
  static constexpr int kCtas = kAlone ? 1 : 2;
  static constexpr int kTile = KB * kSub;
  static constexpr int kOffRing = 0;
  static constexpr int kOffQ = kOffRing + NR * kTile;
  static constexpr int kOffP = kOffQ + KB * kQBox;
  static constexpr int kOffRed = kOffP + 2 * kPBuf;  // [3][4 warps][16] f32
  // the merge's m[16], l[16], o[16][D], then every split's m and l and the
  // weights, [16 splits][16] each, in the first slot: written once every product has completed
  static constexpr int kOffX = kOffRing;
  static constexpr int kXBytes = (2 * kSlots + kSlots * D + 3 * kPagedMaxSplits * kSlots) * 4;
  static_assert(kXBytes <= kTile, "the merge fits a stage");
  static constexpr int kOffBar = kOffRed + 3 * 4 * kSlots * 4;
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
  // lengths and offsets of the sequences, while they are ranked
  static constexpr int kOffSeq = kOffMisc + 16;
  static constexpr int kSeqBytes = (2 * kMaxSortedBatch + 2) * 4;
  // the M = 128 operand of a d = 64 product reads the 16 KB after a V tile as
  // its unused upper half: there is that much after the last slot
  static constexpr int kEnd =
      kOffSeq + kSeqBytes > kOffQ + kSub ? kOffSeq + kSeqBytes : kOffQ + kSub;
  static constexpr int kSmemBytes = kEnd + 1024;  // + alignment slack
  static_assert(kOffP % 1024 == 0, "P^T swizzle atoms must be 1024-byte aligned");
  static_assert(kSmemBytes + 1024 <= 228 * 1024 / kCtas, "CTAs per SM");
};

// Places of K(j) and V(j) in the ring's order, for T tiles.
__device__ __forceinline__ int place_of_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int place_of_v(int j, int T) { return j + 1 < T ? 2 * j + 2 : 2 * j + 1; }

__device__ __forceinline__ void softmax_bar() {
  asm volatile("bar.sync 1, 128;" ::: "memory");
}

// N query slots (of the products' 16) of this thread's lane in tensor memory.
template <int N>
__device__ __forceinline__ void tmem_ld_slots(uint32_t taddr, uint32_t (&r)[N]) {
  static_assert(N == 4 || N == 8 || N == 16, "slots");
  if constexpr (N == 4) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(taddr)
        : "memory");
  } else if constexpr (N == 8) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(taddr)
        : "memory");
  } else {
    tmem_ld16_sync(taddr, r);
  }
}

// U: query slots that the softmax works on (4, 8 or 16); the products have 16
// all the same, those behind U with weights of 0.  At 16 a tile's softmax is
// 2,200 clk, longer than its copies take a lone CTA; at four one sequence of
// 32 K tokens on eight CTAs takes 240 us instead of 275, on 64 of them 43
// instead of 46.
template <int D, int U, bool kAlone>
__global__ void __launch_bounds__(kThreads, FewCfg<D, kAlone>::kCtas)
    sdpa_paged_few_kernel(const __grid_constant__ CUtensorMap tmQ,
                          const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const PagedParams p) {
  using C = FewCfg<D, kAlone>;
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
    mbar_init(bar(C::bQ), 1);
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
    tmem_alloc<kTmemCols>(smem_u32(tmem_slot));
    tmem_relinquish();
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  float* red = reinterpret_cast<float*>(gbase + C::kOffRed);
  float* xm = reinterpret_cast<float*>(gbase + C::kOffX);
  float* xl = xm + kSlots;
  float* xo = xl + kSlots;
  float* xw = xo + kSlots * D;

  // ---- this CTA's (sequence, kv head) and key tiles; the cluster spans the
  // splits.  CTAs start roughly in grid order, so sequences are taken
  // longest-first (up to kMaxSortedBatch of them), ranked by every CTA from
  // its own copy of the lengths: long ones do not trail alone at the end.
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
      off_s[i] = __ldg(p.q_offsets + i);
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
      if (lane == 0) {
        const int tokens = kSlots / p.G;
        mbar_expect_tx(bar(C::bQ), C::KB * 128 * p.G * tokens);
        for (int kb = 0; kb < C::KB; ++kb)
          tma_load_3d(base + C::kOffQ + kb * kQBox, &tmQ, bar(C::bQ), kb * 64, g * p.G, seq.q0);
      }
      PageBoxes<kKeys, C::KB> cur, nxt;
      cur.fetch(p, b, t_begin * kKeys, len, lane);
      int issued = 0;
      // the box of every lane into the ring's next slot; false: gave up
      auto load = [&](const PageBoxes<kKeys, C::KB>& boxes, const CUtensorMap* map, int key0) {
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
          nxt.fetch(p, b, key0 + kKeys, len, lane);
          if (!(ok = load(nxt, &tmK, key0 + kKeys))) break;
        }
        ok = load(cur, &tmV, key0);
        cur = nxt;
      }
      // let every issued copy land before the CTA can exit
      if (lane == 0) {
        paged_wait_drain(bar(C::bQ), 0, p.limit_ns);
        for (int x = max(0, issued - C::NR); x < issued; ++x)
          paged_wait_drain(bar(C::bF(x % C::NR)), (x / C::NR) & 1, p.limit_ns);
      }
    }
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------- MMA issuer
    // Order: S(0), S(1), then per tile j: O(j) once P(j) is published, and
    // S(j+2) into the S buffer that P(j)'s publication has just released.
    if (lane == 0 && T > 0) {
      constexpr uint32_t kIdS = idesc_bf16_f32(kKeys, kSlots, false, false);
      constexpr uint32_t kIdO = idesc_bf16_f32(128, kSlots, true, false);
      const uint64_t q_desc = sdesc_sw128(base + C::kOffQ, 16, 1024);
      const uint64_t k_desc = sdesc_sw128(base + C::kOffRing, 16, 1024);
      const uint64_t v_desc = sdesc_sw128(base + C::kOffRing, kSub, 1024);
      const uint64_t p_desc = sdesc_sw128(base + C::kOffP, 16, 1024);
      auto issue_s = [&](int st, int buf) {
        const uint64_t kd = k_desc + static_cast<uint64_t>((st * C::kTile) >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint64_t koff = static_cast<uint64_t>(((ks >> 2) * kSub + (ks & 3) * 32) >> 4);
          const uint64_t qoff = static_cast<uint64_t>(((ks >> 2) * kQBox + (ks & 3) * 32) >> 4);
          umma_ss(tmem + buf * kSlots, kd + koff, q_desc + qoff, kIdS, ks > 0 ? 1u : 0u);
        }
      };
      auto issue_o = [&](int st, int buf) {
        const uint64_t vd = v_desc + static_cast<uint64_t>((st * C::kTile) >> 4);
        const uint64_t pd = p_desc + static_cast<uint64_t>((buf * kPBuf) >> 4);
#pragma unroll
        for (int ks = 0; ks < kKeys / 16; ++ks) {
          const uint64_t voff = static_cast<uint64_t>((ks * 16 * 128) >> 4);
          const uint64_t poff = static_cast<uint64_t>(((ks >> 2) * 2048 + (ks & 3) * 32) >> 4);
          umma_ss(tmem + 2 * kSlots + buf * kSlots, vd + voff, pd + poff, kIdO,
                  ks > 0 ? 1u : 0u);
        }
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
    const uint32_t tO = tmem + lane_bits + 2 * kSlots;
    const bool o_rows = warp * 32 < D;  // warp-uniform
    const float sl2 = p.scale_log2;
    // the last key each slot sees; -1 for a slot not in use
    int last[U];
#pragma unroll
    for (int q = 0; q < U; ++q)
      last[q] = q >= rows ? -1 : p.causal ? len - seq.n + div_by_group(p, q) : len - 1;
    float m[U], l[U], acc[U], alpha_prev[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      m[q] = -INFINITY;
      l[q] = 0.f;
      acc[q] = 0.f;
      alpha_prev[q] = 1.f;
    }
    // P^T store address of key r: 64-key atom, 16-byte chunk, 2-byte slot
    const int kk = r & 63;
    uint8_t* p_key = gbase + C::kOffP + (r >> 6) * 2048 + (kk & 7) * 2;
    const int chunk = kk >> 3;
    if constexpr (U < kSlots) {
      // weights of the slots behind U, published with the first tile's
      for (int i = threadIdx.x; i < 2 * kPBuf / 16; i += 128)
        *reinterpret_cast<uint4*>(gbase + C::kOffP + i * 16) = make_uint4(0u, 0u, 0u, 0u);
      softmax_bar();
    }
    bool ok = true;
    for (int j = 0; j < T; ++j) {
      const int buf = j & 1;
      const uint32_t par = (j >> 1) & 1;
      const int key = (t_begin + j) * kKeys + r;
      if (!(ok = mbar_wait_warp(bar(C::bS(buf)), par, ctl))) break;
      tc_fence_after();
      uint32_t sr[U];
      tmem_ld_slots<U>(tS + buf * kSlots, sr);
      float s[U];
#pragma unroll
      for (int q = 0; q < U; ++q)
        s[q] = key <= last[q] ? __uint_as_float(sr[q]) * sl2 : -INFINITY;
      float* rb = red + buf * 4 * kSlots;
      {
        float wm[U];
#pragma unroll
        for (int q = 0; q < U; ++q) wm[q] = warp_max_f32(s[q]);
        if (lane == 0) {
          float4* dst = reinterpret_cast<float4*>(rb + warp * kSlots);
#pragma unroll
          for (int i = 0; i < U / 4; ++i)
            dst[i] = make_float4(wm[4 * i], wm[4 * i + 1], wm[4 * i + 2], wm[4 * i + 3]);
        }
      }
      mbar_arrive(bar(C::bRed(buf)));
      if (!(ok = mbar_wait_warp(bar(C::bRed(buf)), par, ctl))) break;
      float alpha[U];
#pragma unroll
      for (int i = 0; i < U / 4; ++i) {
        const float4 a0 = reinterpret_cast<const float4*>(rb)[i];
        const float4 a1 = reinterpret_cast<const float4*>(rb + kSlots)[i];
        const float4 a2 = reinterpret_cast<const float4*>(rb + 2 * kSlots)[i];
        const float4 a3 = reinterpret_cast<const float4*>(rb + 3 * kSlots)[i];
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
          l[q] = fmaf(l[q], alpha[q], pq);
          m[q] = mn;
          s[q] = pq;
        }
      }
      // P^T(j) in bf16 (half a step, 2^-8 of a weight, which the output's own
      // rounding matches): row q, key r, 128-byte swizzle
      uint8_t* pb = p_key + buf * kPBuf;
#pragma unroll
      for (int q = 0; q < U; ++q)
        *reinterpret_cast<__nv_bfloat16*>(pb + (q >> 3) * 1024 + (q & 7) * 128 +
                                          ((chunk ^ (q & 7)) << 4)) = __float2bfloat16_rn(s[q]);
      if ((t_begin + j + 1) * kKeys > len) {
        // V rows behind the length: zero them once the tile has landed (it
        // stays until this tile's product, which waits for the arrive below)
        const int x = place_of_v(j, T);
        if (!(ok = mbar_wait_warp(bar(C::bF(x % C::NR)), (x / C::NR) & 1, ctl))) break;
        if (key >= len) {
          uint8_t* v_row = gbase + C::kOffRing + x % C::NR * C::kTile + r * 128;
#pragma unroll
          for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(v_row + kb * kSub + i * 16) = make_uint4(0u, 0u, 0u, 0u);
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
          uint32_t orr[U];
          tmem_ld_slots<U>(tO + (pj & 1) * kSlots, orr);
#pragma unroll
          for (int q = 0; q < U; ++q)
            acc[q] = fmaf(acc[q], alpha_prev[q], __uint_as_float(orr[q]));
        }
      }
#pragma unroll
      for (int q = 0; q < U; ++q) alpha_prev[q] = alpha[q];
    }
    if (ok && T > 0) {
      const int pj = T - 1;
      if ((ok = mbar_wait_warp(bar(C::bO(pj & 1)), (pj >> 1) & 1, ctl))) {
        tc_fence_after();
        if (o_rows) {
          uint32_t orr[U];
          tmem_ld_slots<U>(tO + (pj & 1) * kSlots, orr);
#pragma unroll
          for (int q = 0; q < U; ++q)
            acc[q] = fmaf(acc[q], alpha_prev[q], __uint_as_float(orr[q]));
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
    float* lsum = red + 2 * 4 * kSlots;
    if (lane == 0) {
      float4* dst = reinterpret_cast<float4*>(lsum + warp * kSlots);
#pragma unroll
      for (int i = 0; i < U / 4; ++i)
        dst[i] = make_float4(l[4 * i], l[4 * i + 1], l[4 * i + 2], l[4 * i + 3]);
    }
    softmax_bar();
    const bool failed = *abort_flag != 0;
    if (failed) *bad_page = 1;  // a failed split spoils the rows
    if (threadIdx.x < kSlots) {
      const int q = threadIdx.x;
      const bool none = failed || q >= U;
      float mq = -INFINITY;
#pragma unroll
      for (int k = 0; k < U; ++k) mq = k == q ? m[k] : mq;
      xm[q] = none ? -INFINITY : mq;
      xl[q] = none ? 0.f
                   : lsum[q] + lsum[kSlots + q] + lsum[2 * kSlots + q] + lsum[3 * kSlots + q];
    }
    if (o_rows && r < D) {
#pragma unroll
      for (int q = 0; q < U; ++q) xo[q * D + r] = acc[q];
    }
  }

  // ---- merge the splits through distributed shared memory: every split's m
  // and l are fetched, each thread works out weights, 2^(m_s - M) / sum, then
  // the outputs, four columns a place, each another remote load
  __syncwarp();
  cluster_sync();  // every split's m, l, O and bad-page flag are in its shared memory
  if (warp < 4) {
    const int S = p.splits;
    float* lm = xw + kPagedMaxSplits * kSlots;
    float* ll = lm + kPagedMaxSplits * kSlots;
    const uint32_t xm_s = smem_u32(xm), xl_s = smem_u32(xl), xo_s = smem_u32(xo);
    const bool bad = any_bad(smem_u32(const_cast<int*>(bad_page)), S);
#pragma unroll 1
    for (int x = threadIdx.x; x < S * kSlots; x += 128) {
      const uint32_t q = x % kSlots, s = x / kSlots;
      lm[x] = ld_cluster_f32(cluster_map(xm_s + 4u * q, s));
      ll[x] = ld_cluster_f32(cluster_map(xl_s + 4u * q, s));
    }
    softmax_bar();
#pragma unroll 1
    for (int x = threadIdx.x; x < S * kSlots; x += 128)
      xw[x] = bad ? 0.f : split_weight(lm + x % kSlots, ll + x % kSlots, kSlots, S, x / kSlots);
    softmax_bar();
    const int total = rows * (D / 4);
    const int per = (total + S - 1) / S;
    const int e0 = split * per;
    const int e1 = min(total, e0 + per);
    const int sharers = merge_sharers(per, S, 128);
#pragma unroll 1
    for (int f0 = e0; f0 < e1; f0 += 128 / sharers) {
      const int e = f0 + static_cast<int>(threadIdx.x) / sharers;
      const int q = e / (D / 4);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      if (e < e1) {
#pragma unroll 2
        for (int s = threadIdx.x % sharers; s < S; s += sharers)
          add_split(o, xo_s + 16u * e, s, xw[s * kSlots + q]);
      }
      sum_sharers(o, sharers);
      if (e < e1 && threadIdx.x % sharers == 0) {
        const int i = div_by_group(p, q);
        const int64_t row = static_cast<int64_t>(seq.q0 + i) * p.H + g * p.G + (q - i * p.G);
        store_out4(p, row * D + (e - q * (D / 4)) * 4, o);
      }
    }
  }
  __syncwarp();
  cluster_sync();  // no CTA leaves while another still reads its shared memory
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc<kTmemCols>(tmem);
  }
}

template <int D, int U, bool kAlone>
cudaError_t launch_as(const PagedSdpaArgs& a, const DeviceCtl& ctl) {
  using C = FewCfg<D, kAlone>;
  CUtensorMap q, k, v;
  if (!paged_tensor_maps(a, D, kSlots / a.G, kKeys, &q, &k, &v)) return cudaErrorInvalidValue;
  const int64_t clusters = static_cast<int64_t>(a.pages.B) * a.pages.kv_heads;
  if (clusters * a.splits > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  auto kern = sdpa_paged_few_kernel<D, U, kAlone>;
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
  e = cudaLaunchKernelEx(&cfg, kern, q, k, v, paged_params(a, ctl));
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D>
cudaError_t launch_impl(PagedSdpaArgs a, const DeviceCtl& ctl) {
  const int64_t clusters = static_cast<int64_t>(a.pages.B) * a.pages.kv_heads;
  if (a.splits == 0)
    a.splits = paged_default_splits(
        clusters, static_cast<int64_t>(a.pages.cols) << a.pages.page_shift, kThreads,
        FewCfg<D, false>::kSmemBytes);
  const bool alone =
      clusters <= paged_resident_clusters(kThreads, FewCfg<D, true>::kSmemBytes, a.splits);
  // the softmax's work per tile goes with the slots: 4, 8 or all 16 of them
  const int64_t rows = static_cast<int64_t>(a.max_new) * a.G;
  if (rows <= 4) return alone ? launch_as<D, 4, true>(a, ctl) : launch_as<D, 4, false>(a, ctl);
  if (rows <= 8) return alone ? launch_as<D, 8, true>(a, ctl) : launch_as<D, 8, false>(a, ctl);
  return alone ? launch_as<D, 16, true>(a, ctl) : launch_as<D, 16, false>(a, ctl);
}

}  // namespace

cudaError_t launch_sdpa_paged_few(const PagedSdpaArgs& a, const DeviceCtl& ctl) {
  return a.pages.d == 64 ? launch_impl<64>(a, ctl) : launch_impl<128>(a, ctl);
}

}  // namespace mha
