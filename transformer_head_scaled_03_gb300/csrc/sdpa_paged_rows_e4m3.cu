// sdpa_paged_rows_e4m3.cu -- paged attention of query tiles over a cache in 8
// bits: chunks of new tokens, or few of them under many shared heads.
//
// Tiles, blocks, splits and the key loop are those of sdpa_paged_rows.cu.  Per
// tile of BN keys:
//   S_t  = Q_t K_codes^T   tcgen05 kind::f8f6f4 over the codes as they lie in
//          the pages; a row of Q over a power of two as two e4m3 parts, one
//          product each into the same accumulator (the 8-bit rate is twice
//          bf16's, so both take the time of one in bf16)
//   s    = S_t f           f = the key's page scale, the row's and the softmax's
//   W_t  = 2^(s + v - R)   v = log2 of the value scale over the CTA's first one
//                          above 0 (a scale of 0: 60 less than the largest so far)
//   O_t += W_t V_codes     kind::f16, W in fp16 from TMEM, the codes in fp16
//          (every one is exact) from shared memory, where warps of their own
//          write them: four beside two query tiles, two beside one
//   l   += sum 2^(s - R) = sum W_t 2^-v, page by page
// R is the running maximum of s + v less kHead, so that a weight has room below
// it: fp16 is off by 2^-11 of a weight, or 2^-25 below 2^-14.
// Weights as two e4m3 parts would spare the converting warps, but cost the
// softmax six instructions a pair of weights instead of one, and it is what the
// loop waits for; a V tile is converted once for all 256 rows of a CTA.  With
// the value scales multiplied in there, in bf16, by two warps, these held the
// loop up: 947 us for the 4,096-token chunks (641 without the conversion).
//
// Bound by the chain softmax, P V, next scores: the tensor pipe is busy 54 % of the
// time, and a softmax warp waits longer for its scores than it works on them.  The
// second part of Q is a tenth of the time (603 us without it, 675 with, when that
// was measured), the conversion 4 % (646).
// Measured: two sequences, 4,096 new of 8,192 tokens, 32 heads on 8, d = 128:
// 675 us, 1.22 PFLOP/s (the bf16 cache: 571); six chunks of 90 to 444 tokens over
// 900 to 7,800 keys, 40 heads on 8: 166 us (146); 16 new tokens each over 30 K
// keys, four sequences: 90 us (101).  The same work in another order of the code
// has taken from 667 to 679 us: the roles share one instruction cache.
#include <math.h>
#include <stdint.h>

#include <cuda_bf16.h>

#include "ptx_e4m3.cuh"
#include "sdpa_paged_rows.cuh"

namespace mha {
namespace {

constexpr int kBlockM = kRowsM;

// Eight of these to a tile at most: pages have 16 rows or more.
constexpr int kPageSlots = 8;

template <int D, int NQT, int NK, int NV, int BN, int kCtas>
struct Rows8Cfg {
  static_assert(D == 64 || D == 128, "head dim");
  static_assert(BN == 64 || BN == 128, "key tile");
  static constexpr int kQPart = kBlockM * D;          // one part of a query tile
  static constexpr int kQTileBytes = 2 * kQPart;
  static constexpr int kTile = BN * D;                // a key or value tile, codes
  static constexpr int kVBlock = BN * 128;            // 64 columns of a value tile in fp16
  static constexpr int kV16Bytes = BN * D * 2;
  static constexpr int NW = 2;                        // value tiles in fp16
  static constexpr int kSoftmaxWarps = 4 * NQT;
  // Two tiles: a warpgroup converts, one copies and issues (two of its warps
  // idle), and both hand registers to the softmax's two: 512 threads start with
  // 128 registers each, and 128 * (2 * 176 + 2 * 80) are as many.  One tile: two
  // warps convert, and nothing is handed over.
  static constexpr bool kHandOver = NQT == 2;
  static constexpr int kConvWarps = kHandOver ? 4 : 2;
  static constexpr int kConvWarp = kSoftmaxWarps;
  static constexpr int kTmaWarp = kConvWarp + kConvWarps;
  static constexpr int kMmaWarp = kTmaWarp + 1;
  static constexpr int kConvThreads = 32 * kConvWarps;
  static constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
  static constexpr int kThreads = kHandOver ? 512 : 32 * (kMmaWarp + 1);
  static constexpr int kTmemNeed = NQT * (BN + D);
  static constexpr uint32_t kTmemCols = kTmemNeed <= 128 ? 128u : kTmemNeed <= 256 ? 256u : 512u;
  static_assert(kTmemNeed <= 512 && kCtas * kTmemCols <= 512, "TMEM budget");
  __host__ __device__ static constexpr uint32_t tS(int t) { return static_cast<uint32_t>(t * BN); }
  __host__ __device__ static constexpr uint32_t tO(int t) { return static_cast<uint32_t>(NQT * BN + t * D); }
  static constexpr int bQ = 0;
  __host__ __device__ static constexpr int bKF(int s) { return 1 + s; }
  __host__ __device__ static constexpr int bKE(int s) { return 1 + NK + s; }
  __host__ __device__ static constexpr int bVF(int s) { return 1 + 2 * NK + s; }
  __host__ __device__ static constexpr int bVE(int s) { return 1 + 2 * NK + NV + s; }
  __host__ __device__ static constexpr int bWF(int s) { return 1 + 2 * NK + 2 * NV + s; }
  __host__ __device__ static constexpr int bWE(int s) { return bWF(0) + NW + s; }
  __host__ __device__ static constexpr int bS(int t) { return bWF(0) + 2 * NW + t; }
  __host__ __device__ static constexpr int bP(int t, int half) { return bS(0) + NQT + 2 * t + half; }
  __host__ __device__ static constexpr int bO(int t) { return bS(0) + 3 * NQT + t; }
  static constexpr int bDrain = bWF(0) + 2 * NW + 4 * NQT;
  static constexpr int bLoaded = bDrain + 1;  // the producer has looked at every page number
  static constexpr int kNumBars = bLoaded + 1;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + NQT * kQTileBytes;
  static constexpr int kOffV = kOffK + NK * kTile;
  static constexpr int kOffW = kOffV + NV * kTile;
  // the merge's partial outputs [NQT * 128][D + 4] f32, over Q and the stages
  // once every product has completed
  static constexpr int kXBytes = NQT * kBlockM * (D + 4) * 4;
  static constexpr int kOffBar = kOffW + NW * kV16Bytes;
  static_assert(kXBytes <= kOffBar, "the merge fits the stages");
  static_assert(kOffK % 1024 == 0 && kOffV % 1024 == 0 && kOffW % 1024 == 0, "swizzle atoms");
  static constexpr int kOffMisc = kOffBar + 8 * kNumBars;
  // of the pages, two tiles longer than the tiles stay (see below): the key
  // scale, log2 of the value scale over the first one, and that ratio's inverse;
  // and the value scales
  static constexpr int NS = NK + 2;
  static constexpr int kOffKs = (kOffMisc + 32 + 15) / 16 * 16;
  static constexpr int kOffVs = kOffKs + NS * kPageSlots * 16;
  static constexpr int kOffQs = kOffVs + NV * kPageSlots * 4;  // scales of the query rows
  static constexpr int kOffM = kOffQs + NQT * kBlockM * 4;     // m, l of every row, f32
  static constexpr int kOffMerge = kOffM + 2 * NQT * kBlockM * 4;
  static constexpr int kShare = NQT * kBlockM + kPagedMaxSplits;
  static constexpr int kSmemBytes = kOffMerge + 3 * kShare * 4 + 1024;  // + alignment slack
  static_assert(kCtas * (kSmemBytes + 1024) <= 228 * 1024, "shared memory");
};

// Four codes as two pairs of fp16.  (The bits moved into place, four instructions
// a pair, took longer: 718 us for the 4,096-token chunks instead of 696.)
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t* v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(i ? w >> 16 : w & 0xffffu), __NV_E4M3);
    v[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Four codes times 0: `nan` where they are NaN.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w, uint32_t nan) {
  return (((w & 0x7f7f7f7fu) + 0x01010101u) >> 7 & 0x01010101u) * nan;
}

// Not to be kept in registers from one use to the next.
__device__ __forceinline__ float4 lds_f32x4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

// kGroup: columns that share a page at least, 32 where pages have as many rows.
template <int D, int NQT, int NK, int NV, int BN, int kCtas, int kGroup>
__global__ void __launch_bounds__(Rows8Cfg<D, NQT, NK, NV, BN, kCtas>::kThreads, kCtas)
    sdpa_paged_rows_e4m3_kernel(const __nv_bfloat16* __restrict__ Q, int64_t q_stride,
                                const __grid_constant__ CUtensorMap tmK,
                                const __grid_constant__ CUtensorMap tmV, const PagedParams p) {
  using C = Rows8Cfg<D, NQT, NK, NV, BN, kCtas>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + C::kOffMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::kOffMisc + 4);
  volatile int* bad_page = reinterpret_cast<volatile int*>(gbase + C::kOffMisc + 8);
  volatile int* pick = reinterpret_cast<volatile int*>(gbase + C::kOffMisc + 16);  // b, head, block
  volatile float* v_first = reinterpret_cast<volatile float*>(gbase + C::kOffMisc + 12);
  float4* k_scales = reinterpret_cast<float4*>(gbase + C::kOffKs);  // [NS][kPageSlots]
  float* v_scales = reinterpret_cast<float*>(gbase + C::kOffVs);  // [NV][kPageSlots]
  float* q_scales = reinterpret_cast<float*>(gbase + C::kOffQs);
  auto bar = [base](int i) -> uint32_t { return base + C::kOffBar + 8u * i; };

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const WaitCtl ctl{abort_flag, p.err, p.limit_ns};
  const int tile_tokens = kBlockM / p.G;
  const int block_tokens = NQT * tile_tokens;

  if (threadIdx.x == 0) {
    mbar_init(bar(C::bQ), NQT * kBlockM);
    for (int s = 0; s < NK; ++s) {
      mbar_init(bar(C::bKF(s)), 1);
      mbar_init(bar(C::bKE(s)), 1);
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(bar(C::bVF(s)), 1);
      mbar_init(bar(C::bVE(s)), C::kConvThreads);
    }
    for (int s = 0; s < C::NW; ++s) {
      mbar_init(bar(C::bWF(s)), C::kConvThreads);
      mbar_init(bar(C::bWE(s)), 1);
    }
    for (int t = 0; t < NQT; ++t) {
      mbar_init(bar(C::bS(t)), 1);
      mbar_init(bar(C::bP(t, 0)), kBlockM);
      mbar_init(bar(C::bP(t, 1)), kBlockM);
      mbar_init(bar(C::bO(t)), 1);
    }
    mbar_init(bar(C::bDrain), 1);
    mbar_init(bar(C::bLoaded), 1);
    *abort_flag = 0;
    *bad_page = 0;
    fence_mbar_init();
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc<C::kTmemCols>(smem_u32(tmem_slot));
    tmem_relinquish();
  }
  if (warp == C::kTmaWarp && lane == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  const int split = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.splits));
  // Q's place, before it is written
  const RowsBlock blk = rows_block<C::kThreads>(p, gbase, pick, block_tokens);
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  const int b = blk.b, g = blk.g, i0 = blk.i0;
  const PagedSeq seq = blk.seq;
  const int len = seq.len;
  // key tiles that query tile t needs: up to its last token's own key
  auto tiles_of = [&](int t) -> int {
    const int i = i0 + t * tile_tokens;
    if (seq.bad_len || i >= seq.n) return 0;
    const int stop =
        p.causal ? len - seq.n + min(seq.n, i + tile_tokens) : len;
    return (stop + BN - 1) / BN;
  };
  // this CTA walks the key tiles [j0, j1), query tile t as far as it needs them
  int n_all = 0;
  for (int t = 0; t < NQT; ++t) n_all = max(n_all, tiles_of(t));
  const int j0 = static_cast<int>(static_cast<int64_t>(n_all) * split / p.splits);
  const int j1 = static_cast<int>(static_cast<int64_t>(n_all) * (split + 1) / p.splits);
  const int n_kv = j1 - j0;
  auto count_of = [&](int t) -> int { return max(0, min(tiles_of(t), j1) - j0); };

  // From here on the roles share no code: a warp that has handed registers over
  // runs none that was compiled for more.
  if (warp >= C::kConvWarp) {
    if constexpr (C::kHandOver) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == C::kTmaWarp) {
      // ------------------------------------------------------------ producer
      // Page numbers are sent for two tiles ahead and the pages' scales one
      // ahead.  A page's row of k_scales is read by the softmax until P_t(j) is published,
      // which S(j + 2) waits for, and its place is written again with the keys
      // of tile j + NS, after S(j + 2) has released theirs.
      if (n_kv > 0) {
        using Boxes = PageBoxes<BN, 1, D>;
        const int32_t* row = table_row(p, b, g);
        auto scales_of = [&](const Boxes& x, float& sk, float& sv) {
          const int64_t at = static_cast<int64_t>(x.page) * p.kv_heads + g;
          sk = x.good(p) ? __ldg(p.k_scale + at) : 0.f;
          sv = x.good(p) ? __ldg(p.v_scale + at) : 0.f;
        };
        Boxes cur, nxt, aft;
        float sk, sv, sk1 = 0.f, sv1 = 0.f;
        aft.mine = false;
        cur.fetch(p, row, j0 * BN, len, lane);
        nxt.fetch(p, row, (j0 + 1) * BN, n_kv > 1 ? len : 0, lane);
        scales_of(cur, sk, sv);
        // value scales count against the first one above 0, so that sums stay in
        // range whatever size they are; those of a sequence lie within 2^100 of each
        // other.  A page of scale 0 (its codes become zeros) takes 2^-60 of the largest
        // so far: its keys count in the sum, and do not raise R above the weights that
        // meet values unless they outweigh those by 2^60; and 2^-72 of the largest
        // weight is still in range.
        float first = 0.f, most = 1.f;
        int k_issued = 0, v_issued = 0;
        for (int j = 0; j < n_kv; ++j) {
          const int ks = j % NK, vs = j % NV;
          const int key0 = (j0 + j) * BN;
          if (cur.bad(p)) {
            *bad_page = 1;
            atomicOr(p.err, kErrPages);
          }
          const uint32_t bytes = cur.bytes(p);
          if (!mbar_wait_warp(bar(C::bKE(ks)), ((j / NK) & 1) ^ 1u, ctl)) break;
          if (first == 0.f) {
            const unsigned some = __ballot_sync(0xffffffffu, sv > 0.f);
            if (some) first = __shfl_sync(0xffffffffu, sv, __ffs(some) - 1);
          }
          const bool none = !(sv > 0.f);
          float ratio = none ? 1.f : fminf(fmaxf(sv / first, 0x1p-100f), 0x1p100f);
          most = fmaxf(most, ratio);  // this lane's
          if (__any_sync(0xffffffffu, none && cur.mine)) {
            // (the order of numbers above 0 is that of their bits)
            most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
            if (none) ratio = most * 0x1p-60f;
          }
          if (lane < kPageSlots) {
            k_scales[j % C::NS * kPageSlots + lane] =
                make_float4(sk, log2f(ratio), 1.f / ratio, 0.f);
          }
          __syncwarp();
          if (lane == 0) mbar_expect_tx(bar(C::bKF(ks)), bytes);
          __syncwarp();
          cur.load(p, &tmK, base + C::kOffK + ks * C::kTile, bar(C::bKF(ks)), key0, g, lane);
          k_issued = j + 1;
          aft.fetch(p, row, key0 + 2 * BN, j + 2 < n_kv ? len : 0, lane);
          scales_of(nxt, sk1, sv1);
          if (!mbar_wait_warp(bar(C::bVE(vs)), ((j / NV) & 1) ^ 1u, ctl)) break;
          if (lane < kPageSlots) v_scales[vs * kPageSlots + lane] = sv;
          __syncwarp();
          if (lane == 0) mbar_expect_tx(bar(C::bVF(vs)), bytes);
          __syncwarp();
          cur.load(p, &tmV, base + C::kOffV + vs * C::kTile, bar(C::bVF(vs)), key0, g, lane);
          v_issued = j + 1;
          cur = nxt;
          nxt = aft;
          sk = sk1;
          sv = sv1;
        }
        __syncwarp();
        if (lane == 0) {
          *v_first = first > 0.f ? first : 1.f;
          mbar_arrive(bar(C::bLoaded));
          // let every issued copy land before the CTA can exit
          for (int j = max(0, k_issued - NK); j < k_issued; ++j)
            paged_wait_drain(bar(C::bKF(j % NK)), (j / NK) & 1, p.limit_ns);
          for (int j = max(0, v_issued - NV); j < v_issued; ++j)
            paged_wait_drain(bar(C::bVF(j % NV)), (j / NV) & 1, p.limit_ns);
        }
      }
    } else if (warp == C::kMmaWarp) {
      // ---------------------------------------------------------- MMA issuer
      // Order per key tile j: PV_0(j), S_0(j+1), PV_1(j), S_1(j+1).  S_t(j+1)
      // overwrites the columns of P_t(j); tcgen05 products of one CTA execute
      // in issue order, so PV_t(j) has read them.
      if (lane == 0 && n_kv > 0) {
        constexpr uint32_t kIdescQK = idesc_e4m3_f32(kBlockM, BN, false, false);
        constexpr uint32_t kIdescPV = idesc_f16_f32(kBlockM, D, false, true);
        const uint64_t q_desc = sdesc_rows<D>(base + C::kOffQ, 16, 8 * D);
        const uint64_t k_desc = sdesc_rows<D>(base + C::kOffK, 16, 8 * D);
        const uint64_t v_desc = sdesc_sw128(base + C::kOffW, C::kVBlock, 1024);
        auto issue_qk = [&](int t, int st) {
          const uint64_t qd = q_desc + static_cast<uint64_t>((t * C::kQTileBytes) >> 4);
          const uint64_t kd = k_desc + static_cast<uint64_t>((st * C::kTile) >> 4);
          const uint32_t d_tmem = tmem + C::tS(t);
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks)
              umma_f8_ss(d_tmem, qd + static_cast<uint64_t>((part * C::kQPart) >> 4) + 2 * ks,
                         kd + 2 * ks, kIdescQK, part + ks > 0 ? 1u : 0u);
        };
        auto issue_pv = [&](int t, int st, int half, uint32_t accumulate) {
          const uint64_t vd = v_desc + static_cast<uint64_t>((st * C::kV16Bytes) >> 4);
          const uint32_t d_tmem = tmem + C::tO(t);
          const uint32_t a_tmem = tmem + C::tS(t);
#pragma unroll
          for (int ks = half * (BN / 32); ks < (half + 1) * (BN / 32); ++ks)
            umma_ts(d_tmem, a_tmem + ks * 8, vd + static_cast<uint64_t>((ks * 16 * 128) >> 4),
                    kIdescPV, ks > 0 ? 1u : accumulate);
        };
        int counts[NQT];
        for (int t = 0; t < NQT; ++t) counts[t] = count_of(t);
        bool ok = mbar_wait(bar(C::bQ), 0, ctl) && mbar_wait(bar(C::bKF(0)), 0, ctl);
        if (ok) {
          tc_fence_after();
#pragma unroll
          for (int t = 0; t < NQT; ++t) {
            if (counts[t] == 0) continue;
            issue_qk(t, 0);
            umma_commit(bar(C::bS(t)));
          }
          umma_commit(bar(C::bKE(0)));
        }
        // A query tile whose last key tile is j gets no S(j + 1); its epilogue
        // runs while the other tile of the CTA walks on.
        for (int j = 0; ok && j < n_kv; ++j) {
          const int w = j % C::NW;
          const bool more = j + 1 < n_kv;
          const int st1 = (j + 1) % NK;
          const uint32_t ph1 = ((j + 1) / NK) & 1;
          if (!(ok = mbar_wait(bar(C::bWF(w)), (j / C::NW) & 1, ctl))) break;
          bool k_ready = false;
#pragma unroll
          for (int t = 0; t < NQT; ++t) {
            if (!ok || j >= counts[t]) continue;
            if (!(ok = mbar_wait(bar(C::bP(t, 0)), j & 1, ctl))) continue;
            tc_fence_after();
            issue_pv(t, w, 0, j > 0 ? 1u : 0u);
            if (!(ok = mbar_wait(bar(C::bP(t, 1)), j & 1, ctl))) continue;
            tc_fence_after();
            issue_pv(t, w, 1, 1u);
            if (j + 1 >= counts[t]) {
              umma_commit(bar(C::bO(t)));
              continue;
            }
            if (!k_ready && !(ok = mbar_wait(bar(C::bKF(st1)), ph1, ctl))) continue;
            k_ready = true;
            issue_qk(t, st1);
            umma_commit(bar(C::bS(t)));
          }
          if (!ok) break;
          if (more) umma_commit(bar(C::bKE(st1)));
          umma_commit(bar(C::bWE(w)));
        }
        // every issued MMA completes before tensor memory is released
        umma_commit(bar(C::bDrain));
        paged_wait_drain(bar(C::bDrain), 0, p.limit_ns);
      }
    } else if (warp < C::kTmaWarp) {
      // ------------------------------------------------- value tiles to fp16
      // A thread takes 16 codes of a key at a time: 16 bytes in, two pieces of 16
      // bytes out.  Rows behind the length hold anything, NaN too, and become
      // zeros, where 0 * NaN would reach the sums; so do codes of scale 0 but
      // for NaN, which an append may have stored beside zeros.
      const int ct = threadIdx.x - 32 * C::kConvWarp;
      constexpr int kPieces = D / 16;  // of a row of codes
      const int c = ct % kPieces;
      const int shift = min(p.page_shift, BN == 128 ? 7 : 6);
      for (int j = 0; j < n_kv; ++j) {
        const int vs = j % NV, w = j % C::NW;
        if (!mbar_wait_warp(bar(C::bVF(vs)), (j / NV) & 1, ctl)) break;
        if (!mbar_wait_warp(bar(C::bWE(w)), ((j / C::NW) & 1) ^ 1u, ctl)) break;
        const uint8_t* from = gbase + C::kOffV + vs * C::kTile;
        uint8_t* to = gbase + C::kOffW + w * C::kV16Bytes + c / 4 * C::kVBlock;
        const int held = len - (j0 + j) * BN;
        // a short loop: unrolled, its instructions push the softmax's out of the
        // instruction cache (1,077 us for the 4,096-token chunks, fully unrolled,
        // where two vectors at a time took 776)
#pragma unroll 1
        for (int r = ct / kPieces; r < BN; r += C::kConvThreads / kPieces) {
          uint4 u = *reinterpret_cast<const uint4*>(from + piece_at<D>(r, c));
          if (r >= held || v_scales[vs * kPageSlots + (r >> shift)] == 0.f) {
            const uint32_t nan = r < held ? 0x7fu : 0u;
            u.x = nan_codes(u.x, nan);
            u.y = nan_codes(u.y, nan);
            u.z = nan_codes(u.z, nan);
            u.w = nan_codes(u.w, nan);
          }
          uint32_t v[8];
          codes_to_half(u.x, v);
          codes_to_half(u.y, v + 2);
          codes_to_half(u.z, v + 4);
          codes_to_half(u.w, v + 6);
          const uint4 lo = make_uint4(v[0], v[1], v[2], v[3]);
          const uint4 hi = make_uint4(v[4], v[5], v[6], v[7]);
          // keys r in rows of 128 bytes (64 columns), 16-byte pieces swizzled;
          // lanes of the other 64 columns (the same banks) take theirs the other
          // way round
          uint8_t* dst = to + r * 128;
          const int p0 = c % 4 * 2, odd = c >> 2;
          *reinterpret_cast<uint4*>(dst + (((p0 + odd) ^ (r & 7)) << 4)) = odd ? hi : lo;
          *reinterpret_cast<uint4*>(dst + (((p0 + 1 - odd) ^ (r & 7)) << 4)) = odd ? lo : hi;
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(C::bWF(w)));
        mbar_arrive(bar(C::bVE(vs)));
      }
    }
    __syncwarp();
    if (p.splits > 1) {
      cluster_sync();
      cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == C::kMmaWarp) tmem_dealloc<C::kTmemCols>(tmem);
  } else {
    if constexpr (C::kHandOver) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    // --------------------------------------------------- softmax warpgroup
    const int t = warp >> 2;
    const int quarter = warp & 3;  // this warp may touch TMEM lanes [32q, 32q+32)
    const int r = quarter * 32 + lane;
    const int i = i0 + t * tile_tokens + div_by_group(p, r);  // this row's token of the sequence
    const int tile_rows = min(tile_tokens, seq.n - i0 - t * tile_tokens) * p.G;
    // rows of this warp that stand for a token (warp-uniform): without any,
    // the warp only takes its part in the hand-overs
    const bool warp_in_use = quarter * 32 < tile_rows;
    const uint32_t lane_bits = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_bits + C::tS(t);
    const uint32_t tO = tmem + lane_bits + C::tO(t);
    const int n_t = count_of(t);
    if (n_kv > 0) {
      // this warp's rows of Q as two parts, four at a time: eight lanes to a
      // row, D / 8 columns each
      constexpr int n = D / 8;
      const int part = lane & 7;
      uint8_t* qt = gbase + C::kOffQ + t * C::kQTileBytes;
      const int64_t head0 = static_cast<int64_t>(g) * p.G;
#pragma unroll 2
      for (int k = 0; k < 8; ++k) {
        const int x = quarter * 32 + k * 4 + (lane >> 3);
        const int tok = div_by_group(p, x);
        const bool here = x < tile_rows && n_t > 0;
        const uint4* from = reinterpret_cast<const uint4*>(
            Q + (seq.q0 + i0 + t * tile_tokens + tok) * q_stride + (head0 + x - tok * p.G) * D +
            part * n);
        float e[n];
        float top = 0.f;
#pragma unroll
        for (int v = 0; v < n / 8; ++v) {
          const uint4 u = here ? __ldg(from + v) : make_uint4(0u, 0u, 0u, 0u);
          const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const float2 f = __bfloat1622float2(h[z]);
            e[8 * v + 2 * z] = f.x;
            e[8 * v + 2 * z + 1] = f.y;
          }
        }
#pragma unroll
        for (int z = 0; z < n; ++z) {
          if (fabsf(e[z]) < INFINITY)
            top = fmaxf(top, fabsf(e[z]));
          else
            e[z] = NAN;  // the row's scores, as infinities would make them in the end
        }
#pragma unroll
        for (int s = 1; s < 8; s <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
        float inv;
        const float scale = part_scale_of(top, &inv);
        if (part == 0) q_scales[t * kBlockM + x] = scale * p.scale_log2;
        uint32_t hi[n / 4], lo[n / 4];
#pragma unroll
        for (int z = 0; z < n / 4; ++z) {
          uint32_t a0, a1, b0, b1;
          two_parts(e[4 * z] * inv, e[4 * z + 1] * inv, 1.f, &a0, &b0);
          two_parts(e[4 * z + 2] * inv, e[4 * z + 3] * inv, 1.f, &a1, &b1);
          hi[z] = a0 | a1 << 16;
          lo[z] = b0 | b1 << 16;
        }
        if constexpr (D == 128) {
          uint8_t* to = qt + piece_at<D>(x, part);
          *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(to + C::kQPart) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        } else {
          uint8_t* to = qt + piece_at<D>(x, part / 2) + (part & 1) * 8;
          *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(to + C::kQPart) = make_uint2(lo[0], lo[1]);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(C::bQ));
      __syncwarp();  // the warp's scales are there
    }
    const float row_scale = n_kv > 0 ? q_scales[t * kBlockM + r] : 0.f;
    // ref: R above, in powers of two as s.  It is raised only when a tile's
    // maximum exceeds it by more than kHead + kRescaleLog2, so that weights stay
    // below 2^14; O and l share it, so O / l is unchanged.
    constexpr float kHead = 6.f, kRescaleLog2 = 8.f;
    float ref = -INFINITY;
    float l = 0.f;
    bool ok = true;
    const int row_last = p.causal ? min(len - 1, len - seq.n + i) : len - 1;
    const int first_last = p.causal ? len - seq.n + i0 + t * tile_tokens : len - 1;
    const int shift = min(p.page_shift, BN == 128 ? 7 : 6);
    for (int j = 0; j < n_t; ++j) {
      const int k0 = (j0 + j) * BN;
      if (!(ok = mbar_wait_warp(bar(C::bS(t)), j & 1, ctl))) break;
      tc_fence_after();
      if (warp_in_use) {
        float x[BN];
        {
          uint32_t s[BN];
#pragma unroll
          for (int c = 0; c < BN; c += 32)
            tmem_ld32(tS + c, *reinterpret_cast<uint32_t(*)[32]>(&s[c]));
          tmem_ld_wait(s);
#pragma unroll
          for (int c = 0; c < BN; ++c) x[c] = __uint_as_float(s[c]);
        }
        // columns past the row's last visible key (tile-uniform test)
        if (k0 + BN - 1 > first_last || k0 + BN > len) {
          const int last = row_last - k0;
#pragma unroll
          for (int c = 0; c < BN; ++c) x[c] = c <= last ? x[c] : -INFINITY;
        }
        // kGroup columns share a page, so its scales: four groups' stay in
        // registers, eight are loaded where they are used.  A factor of 0 counts
        // as the smallest normal number: 0 times the -inf of a hidden key is none.
        const float4* ks = k_scales + j % C::NS * kPageSlots;
        float4 held[kGroup == 32 ? BN / 32 : 1];
        if constexpr (kGroup == 32) {
#pragma unroll
          for (int c = 0; c < BN / 32; ++c) {
            held[c] = ks[(32 * c) >> shift];
            held[c].x = fmaxf(held[c].x * row_scale, 0x1p-126f);
          }
        }
        auto scales_at = [&](int c) {
          if constexpr (kGroup == 32) return held[c / 32];
          float4 s = lds_f32x4(smem_u32(ks + (c >> shift)));
          s.x = fmaxf(s.x * row_scale, 0x1p-126f);
          return s;
        };
        float mt = -INFINITY;
#pragma unroll
        for (int c = 0; c < BN; c += 16) {
          const float a = fmax3(fmax3(x[c], x[c + 1], x[c + 2]), x[c + 3], x[c + 4]);
          const float d = fmax3(fmax3(x[c + 5], x[c + 6], x[c + 7]), x[c + 8], x[c + 9]);
          const float e = fmax3(fmax3(x[c + 10], x[c + 11], x[c + 12]), x[c + 13], x[c + 14]);
          const float4 s = scales_at(c);
          mt = fmaxf(mt, fmaf(fmaxf(fmax3(a, d, e), x[c + 15]), s.x, s.y));
        }
        float alpha = 1.f;
        if (mt > ref && (ref == -INFINITY || mt - ref > kHead + kRescaleLog2)) {
          // 0 when ref = -inf; in two steps for l, which keys of scale 0 may have
          // made as large as the reference moves beyond fp32
          const float half = ex2_approx(0.5f * (ref - (mt - kHead)));
          alpha = half * half;
          ref = mt - kHead;
          l = l * half * half;
        }
        // Rescale the partial output when the reference moved.  P.V of the
        // previous tile is complete: it was issued before this tile's S,
        // whose commit covers it.
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          // rarely, and eight columns at a time: the scores hold the registers
#pragma unroll 1
          for (int cb = 0; cb < D; cb += 8) {
            uint32_t o[8];
            tmem_ld8_sync(tO + cb, o);
#pragma unroll
            for (int c = 0; c < 8; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
            tmem_st8(tO + cb, o);
          }
        }
        const float rb = ref == -INFINITY ? 0.f : ref;
        // W in fp16, published in two halves, so that the products of the first
        // run under the exponentials of the second; l sums the unrounded weights
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pk[BN / 4];
#pragma unroll
          for (int c = 0; c < BN / 32; ++c) {
            const int group = half * (BN / 32) + c;
            const float4 s = scales_at(16 * group);
            const float2 f2 = make_float2(s.x, s.x);
            const float2 shift2 = make_float2(s.y - rb, s.y - rb);
            float2 acc = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int at = 16 * group + 2 * k;
              const float2 e = ffma2(make_float2(x[at], x[at + 1]), f2, shift2);
              const float2 w = make_float2(ex2_approx(e.x), ex2_approx(e.y));
              acc = fadd2(acc, w);
              pk[8 * c + k] = pack_f16x2(w.x, w.y);
            }
            l = fmaf(acc.x + acc.y, s.z, l);
          }
          if constexpr (BN == 128)
            tmem_st32(tS + half * 32, pk);
          else
            tmem_st16(tS + half * 16, pk);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(bar(C::bP(t, half)));
        }
      } else {
        mbar_arrive(bar(C::bP(t, 0)));
        mbar_arrive(bar(C::bP(t, 1)));
      }
    }
    // ------------------------------------------------------------ epilogue
    bool have = ok && n_t > 0;
    if (have) {
      have = mbar_wait_warp(bar(C::bO(t)), 0, ctl);
      tc_fence_after();
    }
    bool zero = !have;  // warp-uniform
    if (n_kv > 0) {
      if (!mbar_wait_warp(bar(C::bLoaded), 0, ctl)) zero = true;
      if (*bad_page) zero = true;
    }
    const bool some = have && l != 0.f;                // NaN stays NaN
    const float inv_l = some ? *v_first / l : 0.f;
    if (p.splits > 1) {
      // the partial outputs go where Q and the stages were: not before every
      // product of the CTA has read them
      for (int o = 0; o < NQT; ++o)
        if (o != t && count_of(o) > 0) ok = mbar_wait_warp(bar(C::bO(o)), 0, ctl) && ok;
      float* xo = reinterpret_cast<float*>(gbase) + (t * kBlockM + r) * (D + 4);
      float* xm = reinterpret_cast<float*>(gbase + C::kOffM);
      if (!ok || (n_t > 0 && !have)) *bad_page = 1;  // a failed split spoils the row
      // a split's outputs are merged as they would be alone, with the logarithm of
      // its sum: the references of splits, which hold value scales, may lie further
      // apart than fp32 reaches
      xm[t * kBlockM + r] = some ? ref + __log2f(l) : -INFINITY;
      xm[(NQT + t) * kBlockM + r] = some ? 1.f : 0.f;
      if (have && warp_in_use) {
#pragma unroll
        for (int cb = 0; cb < D / 32; ++cb) {
          uint32_t o[32];
          tmem_ld32(tO + cb * 32, o);
          tmem_ld_wait(o);
#pragma unroll
          for (int c = 0; c < 8; ++c)
            *reinterpret_cast<float4*>(xo + cb * 32 + 4 * c) =
                make_float4(__uint_as_float(o[4 * c]) * inv_l, __uint_as_float(o[4 * c + 1]) * inv_l,
                            __uint_as_float(o[4 * c + 2]) * inv_l, __uint_as_float(o[4 * c + 3]) * inv_l);
        }
      }
    } else if (warp_in_use) {
      const int64_t row0 = static_cast<int64_t>(seq.q0 + i0 + t * tile_tokens) * p.H + g * p.G;
      rows_store<D>(p, tO, zero, inv_l, quarter, tile_rows, row0,
                    gbase + C::kOffQ + t * C::kQTileBytes);
    }
    __syncwarp();
    if (p.splits > 1) {
      cluster_sync();  // every split's m, l, O and bad-page flag are in its shared memory
      rows_merge<D, NQT, C::kSoftmaxThreads>(p, seq, g, i0, split, tile_tokens, base,
                                             base + C::kOffM,
                                             reinterpret_cast<float*>(gbase + C::kOffMerge),
                                             bad_page);
      __syncwarp();
      cluster_sync();  // no CTA leaves while another still reads its shared memory
    }
    tc_fence_before();
    __syncthreads();
  }
}

template <int D, int NQT, int NK, int NV, int BN, int kCtas, int kGroup>
cudaError_t launch_as(PagedSdpaArgs a, const DeviceCtl& ctl) {
  using C = Rows8Cfg<D, NQT, NK, NV, BN, kCtas>;
  CUtensorMap k, v;
  if (!paged_tensor_maps_e4m3(a, D, BN, &k, &v)) return cudaErrorInvalidValue;
  const int64_t blocks = rows_block_bound(a, NQT * (kBlockM / a.G));
  if (a.splits == 0)
    a.splits = paged_default_splits(
        blocks, static_cast<int64_t>(a.pages.cols) << a.pages.page_shift, C::kThreads, C::kSmemBytes);
  if (blocks * a.splits > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  auto kern = sdpa_paged_rows_e4m3_kernel<D, NQT, NK, NV, BN, kCtas, kGroup>;
  static std::atomic<uint64_t> attributes_set{0};
  cudaError_t e = paged_kernel_attributes(reinterpret_cast<const void*>(kern), C::kSmemBytes,
                                          &attributes_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks * a.splits));
  cfg.blockDim = dim3(C::kThreads);
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

// Eight pages to a tile cost the two-tile kernels 4 to 5 % (4,096-token chunks 704
// us instead of 674; chunks of 90 to 444 tokens 175 instead of 166), so pages of 32
// rows or more take a kernel of their own; of the one-tile kernels, which wait
// for memory, it is nothing.
template <int D>
cudaError_t launch_two(const PagedSdpaArgs& a, const DeviceCtl& ctl) {
  constexpr int NK = D == 64 ? 4 : 3, NV = D == 64 ? 3 : 2;
  return a.pages.page_shift >= 5 ? launch_as<D, 2, NK, NV, 128, 1, 32>(a, ctl)
                                 : launch_as<D, 2, NK, NV, 128, 1, 16>(a, ctl);
}

}  // namespace

cudaError_t launch_sdpa_paged_rows_e4m3(const PagedSdpaArgs& a, const DeviceCtl& ctl) {
  // Two query tiles per CTA share the key tiles and the converted value tiles,
  // and keep the tensor core busy during one tile's softmax: taken when a
  // sequence can have two tiles of new tokens.  One tile: two CTAs per SM, with
  // 64-key tiles, whose scores fit 128 registers (at d = 128 but for 136 bytes of
  // spills; two tiles over pages of 16 rows spill 36).
  if (a.max_new > kBlockM / a.G)
    return a.pages.d == 64 ? launch_two<64>(a, ctl) : launch_two<128>(a, ctl);
  return a.pages.d == 64 ? launch_as<64, 1, 4, 4, 64, 2, 16>(a, ctl)
                         : launch_as<128, 1, 3, 2, 64, 2, 16>(a, ctl);
}

}  // namespace mha
