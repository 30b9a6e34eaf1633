// sdpa_paged_rows.cu -- paged attention of query tiles: chunks of new tokens,
// or few of them under many shared heads.
//
// A tile is 128 query rows of one (sequence, kv head): floor(128 / G) tokens
// times the G query heads that share the kv head, row = token * G + head, so
// that a short chunk still fills the tensor core's M side and every page is
// read once for all of them.  Per tile of BN keys, gathered from its pages by
// TMA boxes (one lane of the producer warp per box):
//   S_t  = Q_t K_j^T           tcgen05.mma, accumulator in TMEM
//   P_t  = 2^(S_t*c - m*c)     softmax warps, thread r owns query row r; P in
//                              bf16 over S's columns
//   O_t += P_t V_j             tcgen05.mma, A = P_t from TMEM
// A CTA takes NQT tiles, which share the key tiles, and, when there are few
// CTAs, only a share of the keys: the CTAs of a thread-block cluster split
// them and merge exactly (o = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s).
//
// The rows of the last page behind the sequence's length hold anything, NaN
// too: their scores are replaced, and their V rows zeroed in shared memory
// before the product, where 0 * NaN would reach the sums.
//
// Bound by the chain softmax -> P V -> next S of a tile: with two tiles in
// turn a 128-key step of 256 rows takes 2,950 clk where the tensor core needs
// 2,048 (d = 128; 94 % of the measured burst rate of a large library product).
// Measured: two sequences, 4,096 new of 8,192 tokens, 32 heads on 8: 594 us,
// 1.39 PFLOP/s; a CTA's set-up and output are a tenth of it.  Six chunks of 90
// to 444 tokens over 900 to 7,800 keys, 40 heads on 8: 149 us, 1.06 PFLOP/s:
// 256 blocks of 6 to 61 steps on 152 SMs; splitting their keys costs more than
// it evens out (170 us).  16 new tokens each over 30 K keys, four sequences:
// 101 us, 4.9 TB/s, HBM and the one-tile form's exposed chain together.
#include <math.h>
#include <stdint.h>

#include <cuda_bf16.h>

#include "sdpa_paged.cuh"

namespace mha {
namespace {

constexpr int kBlockM = 128;    // query rows per tile = TMEM lanes
constexpr int kSub = 128 * 128;  // bytes of a 128-row x 64-column bf16 block
constexpr int kMaxSorted = 256;  // sequences that a CTA ranks by length

// BN = keys per K/V tile (128, or 64 to fit two CTAs of two d = 64 tiles in
// tensor memory).
template <int D, int NQT, int NST, int BN>
struct RowsCfg {
  static_assert(D == 64 || D == 128, "head dim");
  static_assert(BN == 64 || BN == 128, "key tile");
  static constexpr int KB = D / 64;
  static constexpr int kQTileBytes = KB * kSub;
  static constexpr int kKVBlock = BN * 128;
  static constexpr int kKVTileBytes = KB * kKVBlock;
  static constexpr int kSoftmaxWarps = 4 * NQT;
  static constexpr int kTmaWarp = kSoftmaxWarps;
  static constexpr int kMmaWarp = kSoftmaxWarps + 1;
  static constexpr int kThreads = 32 * (kSoftmaxWarps + 2);
  static constexpr int kTmemNeed = NQT * (BN + D);
  static constexpr uint32_t kTmemCols = kTmemNeed <= 128 ? 128u : kTmemNeed <= 256 ? 256u : 512u;
  static_assert(kTmemNeed <= 512, "TMEM budget");
  // two CTAs per SM where tensor memory and shared memory allow: one's set-up
  // and merge run under the other's products
  static constexpr int kMinBlocks = D == 64 || NQT == 1 ? 2 : 1;
  __host__ __device__ static constexpr uint32_t tS(int t) { return static_cast<uint32_t>(t * BN); }
  __host__ __device__ static constexpr uint32_t tO(int t) { return static_cast<uint32_t>(NQT * BN + t * D); }
  static constexpr int bQ = 0;
  __host__ __device__ static constexpr int bKF(int s) { return 1 + s; }
  __host__ __device__ static constexpr int bKE(int s) { return 1 + NST + s; }
  __host__ __device__ static constexpr int bVF(int s) { return 1 + 2 * NST + s; }
  __host__ __device__ static constexpr int bVE(int s) { return 1 + 3 * NST + s; }
  __host__ __device__ static constexpr int bS(int t) { return 1 + 4 * NST + t; }
  __host__ __device__ static constexpr int bP(int t) { return 1 + 4 * NST + NQT + t; }
  __host__ __device__ static constexpr int bO(int t) { return 1 + 4 * NST + 2 * NQT + t; }
  static constexpr int bDrain = 1 + 4 * NST + 3 * NQT;
  static constexpr int bLoaded = bDrain + 1;  // the producer has looked at every page number
  static constexpr int kNumBars = bLoaded + 1;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + NQT * kQTileBytes;
  static constexpr int kOffV = kOffK + NST * kKVTileBytes;
  // the merge's partial outputs [NQT * 128][D + 4] f32, over Q and the key/value
  // stages once every product has completed (rows 16 bytes apart modulo 128:
  // no bank conflicts)
  static constexpr int kXRow = D + 4;
  static constexpr int kXBytes = NQT * kBlockM * kXRow * 4;
  static constexpr int kOffBar = kOffV + NST * kKVTileBytes;
  static_assert(kXBytes <= kOffBar, "the merge fits the stages");
  static constexpr int kOffMisc = kOffBar + 8 * kNumBars;
  static constexpr int kOffM = kOffMisc + 32;  // m, l of every row, f32
  static constexpr int kOffW = kOffM + 2 * NQT * kBlockM * 4;
  // of this CTA's share of the rows, for every split: weights, m, l
  static constexpr int kShare = NQT * kBlockM + kPagedMaxSplits;
  static constexpr int kWBytes = 3 * kShare * 4;
  static constexpr int kSmemBytes = kOffW + kWBytes + 1024;  // + alignment slack
  static_assert(kSmemBytes <= 232448, "shared memory");
};

template <int D, int NQT, int NST, int BN>
__global__ void __launch_bounds__(RowsCfg<D, NQT, NST, BN>::kThreads,
                                  RowsCfg<D, NQT, NST, BN>::kMinBlocks)
    sdpa_paged_rows_kernel(const __grid_constant__ CUtensorMap tmQ,
                           const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const PagedParams p) {
  using C = RowsCfg<D, NQT, NST, BN>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + C::kOffMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::kOffMisc + 4);
  volatile int* bad_page = reinterpret_cast<volatile int*>(gbase + C::kOffMisc + 8);
  volatile int* pick = reinterpret_cast<volatile int*>(gbase + C::kOffMisc + 16);  // b, head, block
  auto bar = [base](int i) -> uint32_t { return base + C::kOffBar + 8u * i; };

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const WaitCtl ctl{abort_flag, p.err, p.limit_ns};
  const int tile_tokens = kBlockM / p.G;
  const int block_tokens = NQT * tile_tokens;

  if (threadIdx.x == 0) {
    mbar_init(bar(C::bQ), 1);
    for (int s = 0; s < NST; ++s) {
      mbar_init(bar(C::bKF(s)), 1);
      mbar_init(bar(C::bKE(s)), 1);
      mbar_init(bar(C::bVF(s)), 1);
      mbar_init(bar(C::bVE(s)), 1);
    }
    for (int t = 0; t < NQT; ++t) {
      mbar_init(bar(C::bS(t)), 1);
      mbar_init(bar(C::bP(t)), kBlockM);
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
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  // ---- which (sequence, kv head, block of tokens) this CTA computes: blocks
  // are numbered sequence by sequence, longest first (CTAs start in grid
  // order, so long ones do not trail alone at the end; up to kMaxSorted
  // sequences, ranked by every CTA itself); in a sequence head by head (a
  // head's blocks run at about the same time and share its pages in L2), in a
  // head from the last tokens to the first, which see fewer keys.
  int* lens_s = reinterpret_cast<int*>(gbase);  // Q's place, before it is loaded
  int* off_s = lens_s + kMaxSorted;
  int* order_s = off_s + kMaxSorted + 1;
  const bool sorted = p.B > 1 && p.B <= kMaxSorted;
  if (sorted) {
    for (int i = threadIdx.x; i <= p.B; i += C::kThreads) {
      off_s[i] = __ldg(p.q_offsets + i);
      if (i < p.B) lens_s[i] = __ldg(p.kv_len + i);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.B; c += C::kThreads) {
      const int lc = lens_s[c];
      int rank = 0;
#pragma unroll 8
      for (int o = 0; o < p.B; ++o) {
        const int lo = lens_s[o];
        rank += (lo > lc || (lo == lc && o < c)) ? 1 : 0;
      }
      order_s[rank] = c;
    }
    __syncthreads();
  }
  auto seq_of = [&](int i) {
    return sorted ? paged_seq_of(p, off_s[i], off_s[i + 1], lens_s[i]) : paged_seq(p, i);
  };
  const int split = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.splits));
  if (warp == 0) {
    int64_t rest = blockIdx.x / static_cast<unsigned>(p.splits);
    int found = -1, head = 0, blk = 0;
    for (int b0 = 0; b0 < p.B && found < 0; b0 += 32) {
      int seq_b = b0 + lane;
      int n = 0;
      if (seq_b < p.B) {
        if (sorted) seq_b = order_s[seq_b];
        n = seq_of(seq_b).n;
      }
      const int blocks = (n + block_tokens - 1) / block_tokens;
      const int64_t mine = static_cast<int64_t>(blocks) * p.kv_heads;
      int64_t incl = mine;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, s);
        if (lane >= s) incl += up;
      }
      const unsigned in = __ballot_sync(0xffffffffu, rest < incl);
      if (in) {
        const int src = __ffs(in) - 1;
        const int64_t off = __shfl_sync(0xffffffffu, rest - (incl - mine), src);
        const int nb = __shfl_sync(0xffffffffu, blocks, src);
        found = __shfl_sync(0xffffffffu, seq_b, src);
        head = static_cast<int>(off / nb);
        blk = nb - 1 - static_cast<int>(off - static_cast<int64_t>(head) * nb);
      } else {
        rest -= __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    // the first CTA reports bad offsets and lengths, for all sequences
    if (blockIdx.x == 0) {
      for (int b = lane; b < p.B; b += 32) {
        const PagedSeq s = seq_of(b);
        if (s.bad_offsets || s.bad_len) atomicOr(p.err, kErrPages);
      }
    }
    if (lane == 0) {
      pick[0] = found;
      pick[1] = head;
      pick[2] = blk;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  const int b = pick[0];
  const int g = pick[1];
  const int i0 = pick[2] * block_tokens;  // the block's first token of the sequence
  PagedSeq seq{};
  if (b >= 0) seq = seq_of(b);
  if (sorted) {
    fence_proxy_async_smem();  // the copies that follow write over the sequences
    __syncthreads();
  }
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

  if (warp == C::kTmaWarp) {
    // ------------------------------------------------------------ producer
    if (n_kv > 0) {
      if (lane == 0) {
        mbar_expect_tx(bar(C::bQ), NQT * C::KB * 128 * p.G * tile_tokens);
        for (int t = 0; t < NQT; ++t)
          for (int kb = 0; kb < C::KB; ++kb)
            tma_load_3d(base + C::kOffQ + (t * C::KB + kb) * kSub, &tmQ, bar(C::bQ), kb * 64,
                        g * p.G, seq.q0 + i0 + t * tile_tokens);
      }
      PageBoxes<BN, C::KB> cur, nxt;
      cur.fetch(p, b, j0 * BN, len, lane);
      int k_issued = 0, v_issued = 0;
      for (int j = 0; j < n_kv; ++j) {
        const int st = j % NST;
        const uint32_t ph = (j / NST) & 1;
        const int key0 = (j0 + j) * BN;
        if (cur.bad(p)) {
          *bad_page = 1;
          atomicOr(p.err, kErrPages);
        }
        const uint32_t bytes = cur.bytes(p);
        if (!mbar_wait_warp(bar(C::bKE(st)), ph ^ 1u, ctl)) break;
        if (lane == 0) mbar_expect_tx(bar(C::bKF(st)), bytes);
        __syncwarp();
        cur.load(p, &tmK, base + C::kOffK + st * C::kKVTileBytes, bar(C::bKF(st)), key0, g, lane);
        k_issued = j + 1;
        if (j + 1 < n_kv) nxt.fetch(p, b, key0 + BN, len, lane);
        if (!mbar_wait_warp(bar(C::bVE(st)), ph ^ 1u, ctl)) break;
        if (lane == 0) mbar_expect_tx(bar(C::bVF(st)), bytes);
        __syncwarp();
        cur.load(p, &tmV, base + C::kOffV + st * C::kKVTileBytes, bar(C::bVF(st)), key0, g, lane);
        v_issued = j + 1;
        cur = nxt;
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(C::bLoaded));
        // let every issued copy land before the CTA can exit
        paged_wait_drain(bar(C::bQ), 0, p.limit_ns);
        for (int j = max(0, k_issued - NST); j < k_issued; ++j)
          paged_wait_drain(bar(C::bKF(j % NST)), (j / NST) & 1, p.limit_ns);
        for (int j = max(0, v_issued - NST); j < v_issued; ++j)
          paged_wait_drain(bar(C::bVF(j % NST)), (j / NST) & 1, p.limit_ns);
      }
    }
  } else if (warp == C::kMmaWarp) {
    // ---------------------------------------------------------- MMA issuer
    // Order per key tile j: PV_0(j), S_0(j+1), PV_1(j), S_1(j+1).  S_t(j+1)
    // overwrites the columns of P_t(j); tcgen05 products of one CTA execute
    // in issue order, so PV_t(j) has read them.
    if (lane == 0 && n_kv > 0) {
      constexpr uint32_t kIdescQK = idesc_bf16_f32(kBlockM, BN, false, false);
      constexpr uint32_t kIdescPV = idesc_bf16_f32(kBlockM, D, false, true);
      const uint64_t q_desc = sdesc_sw128(base + C::kOffQ, 16, 1024);
      const uint64_t k_desc = sdesc_sw128(base + C::kOffK, 16, 1024);
      const uint64_t v_desc = sdesc_sw128(base + C::kOffV, C::kKVBlock, 1024);
      auto issue_qk = [&](int t, int st) {
        const uint64_t qd = q_desc + static_cast<uint64_t>((t * C::kQTileBytes) >> 4);
        const uint64_t kd = k_desc + static_cast<uint64_t>((st * C::kKVTileBytes) >> 4);
        const uint32_t d_tmem = tmem + C::tS(t);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint64_t qoff = static_cast<uint64_t>(((ks >> 2) * kSub + (ks & 3) * 32) >> 4);
          const uint64_t koff =
              static_cast<uint64_t>(((ks >> 2) * C::kKVBlock + (ks & 3) * 32) >> 4);
          umma_ss(d_tmem, qd + qoff, kd + koff, kIdescQK, ks > 0 ? 1u : 0u);
        }
      };
      auto issue_pv = [&](int t, int st, uint32_t accumulate) {
        const uint64_t vd = v_desc + static_cast<uint64_t>((st * C::kKVTileBytes) >> 4);
        const uint32_t d_tmem = tmem + C::tO(t);
        const uint32_t a_tmem = tmem + C::tS(t);
#pragma unroll
        for (int ks = 0; ks < BN / 16; ++ks)
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
        const int st = j % NST;
        const uint32_t ph = (j / NST) & 1;
        const bool more = j + 1 < n_kv;
        const int st1 = (j + 1) % NST;
        const uint32_t ph1 = ((j + 1) / NST) & 1;
        if (!(ok = mbar_wait(bar(C::bVF(st)), ph, ctl))) break;
        bool k_ready = false;
#pragma unroll
        for (int t = 0; t < NQT; ++t) {
          if (!ok || j >= counts[t]) continue;
          if (!(ok = mbar_wait(bar(C::bP(t)), j & 1, ctl))) continue;
          tc_fence_after();
          issue_pv(t, st, j > 0 ? 1u : 0u);
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
        umma_commit(bar(C::bVE(st)));
      }
      // every issued MMA completes before tensor memory is released
      umma_commit(bar(C::bDrain));
      paged_wait_drain(bar(C::bDrain), 0, p.limit_ns);
    }
  } else {
    // --------------------------------------------------- softmax warpgroup
    const int t = warp >> 2;
    const int quarter = warp & 3;  // this warp may touch TMEM lanes [32q, 32q+32)
    const int r = quarter * 32 + lane;
    const int i = i0 + t * tile_tokens + div_by_group(p, r);  // this row's token of the sequence
    const int tile_rows = min(tile_tokens, seq.n - i0 - t * tile_tokens) * p.G;
    const bool in_use = r < tile_rows;
    // rows of this warp that stand for a token (warp-uniform): without any,
    // the warp only takes its part in the hand-overs
    const bool warp_in_use = quarter * 32 < tile_rows;
    const uint32_t lane_bits = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_bits + C::tS(t);
    const uint32_t tO = tmem + lane_bits + C::tO(t);
    const float sl2 = p.scale_log2;
    // m_ref: the reference that p = 2^((s - m_ref) * sl2) is taken against.
    // It is raised only when a tile's maximum exceeds it by more than
    // kRescaleLog2; O and l share it, so O / l is unchanged.
    constexpr float kRescaleLog2 = 8.f;
    float m_ref = -INFINITY;
    float l = 0.f;
    bool ok = true;
    const int n_t = count_of(t);
    const int row_last = p.causal ? min(len - 1, len - seq.n + i) : len - 1;
    const int first_last = p.causal ? len - seq.n + i0 + t * tile_tokens : len - 1;
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
        // tile maximum: eight independent 3-input max chains, then combine
        float m8[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) m8[c] = fmax3(x[c], x[8 + c], x[16 + c]);
#pragma unroll
        for (int c = 24; c < BN - 8; c += 16)
#pragma unroll
          for (int k = 0; k < 8; ++k) m8[k] = fmax3(m8[k], x[c + k], x[c + 8 + k]);
#pragma unroll
        for (int c = 0; c < 8; ++c) m8[c] = fmaxf(m8[c], x[BN - 8 + c]);
        const float mt = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]),
                               fmaxf(m8[6], m8[7]));
        float alpha = 1.f;
        if (mt > m_ref && (m_ref == -INFINITY || (mt - m_ref) * sl2 > kRescaleLog2)) {
          alpha = ex2_approx((m_ref - mt) * sl2);  // 0 when m_ref = -inf
          m_ref = mt;
          l *= alpha;
        }
        const float mb = m_ref == -INFINITY ? 0.f : m_ref * sl2;
        const float2 scale2 = make_float2(sl2, sl2);
        const float2 shift2 = make_float2(-mb, -mb);
        float2 acc[4];
        uint32_t pk[BN / 2];
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[c] = make_float2(0.f, 0.f);
        // P in bf16: half a step, 2^-8 of a weight; l sums the unrounded ones
#pragma unroll
        for (int c = 0; c < BN / 2; ++c) {
          const float2 e = ffma2(make_float2(x[2 * c], x[2 * c + 1]), scale2, shift2);
          const float2 pp = make_float2(ex2_approx(e.x), ex2_approx(e.y));
          acc[c & 3] = fadd2(acc[c & 3], pp);
          pk[c] = pack_bf16x2(pp.x, pp.y);
        }
        const float2 a = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
        l += a.x + a.y;
#pragma unroll
        for (int c = 0; c < BN / 2; c += 32)
          tmem_st32(tS + c, *reinterpret_cast<const uint32_t(*)[32]>(&pk[c]));
        // Rescale the partial output when the reference moved.  P.V of the
        // previous tile is complete: it was issued before this tile's S,
        // whose commit covers it.
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
          for (int cb = 0; cb < D / 32; ++cb) {
            uint32_t o[32];
            tmem_ld32(tO + cb * 32, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
            tmem_st32(tO + cb * 32, o);
          }
        }
        tmem_st_wait();
      }
      if (k0 + BN > len) {
        // V rows behind the length: zero them once the tile has landed (it
        // stays until this tile's product, which waits for the arrive below;
        // the other query tile's group may write the same zeros)
        const int st = j % NST;
        if (!(ok = mbar_wait_warp(bar(C::bVF(st)), (j / NST) & 1, ctl))) break;
        if (r < BN && k0 + r >= len) {
          uint8_t* v_row = gbase + C::kOffV + st * C::kKVTileBytes + r * 128;
#pragma unroll
          for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
            for (int c = 0; c < 8; ++c)
              *reinterpret_cast<uint4*>(v_row + kb * C::kKVBlock + c * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      tc_fence_before();
      mbar_arrive(bar(C::bP(t)));
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
    if (p.splits > 1) {
      // the partial outputs go where Q and the stages were: not before every
      // product of the CTA has read them
      for (int o = 0; o < NQT; ++o)
        if (o != t && count_of(o) > 0) ok = mbar_wait_warp(bar(C::bO(o)), 0, ctl) && ok;
      float* xo = reinterpret_cast<float*>(gbase) + (t * kBlockM + r) * C::kXRow;
      float* xm = reinterpret_cast<float*>(gbase + C::kOffM);
      if (!ok || (n_t > 0 && !have)) *bad_page = 1;  // a failed split spoils the row
      xm[t * kBlockM + r] = have && m_ref != -INFINITY ? m_ref * sl2 : -INFINITY;
      xm[(NQT + t) * kBlockM + r] = have ? l : 0.f;
      if (have && warp_in_use) {
#pragma unroll
        for (int cb = 0; cb < D / 32; ++cb) {
          uint32_t o[32];
          tmem_ld32(tO + cb * 32, o);
          tmem_ld_wait(o);
#pragma unroll
          for (int c = 0; c < 8; ++c)
            *reinterpret_cast<uint4*>(xo + cb * 32 + 4 * c) =
                make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
        }
      }
    } else if (warp_in_use) {
      const float inv_l = !zero && l != 0.f ? 1.f / l : 0.f;  // NaN stays NaN
      const int rows_here = min(32, tile_rows - quarter * 32);
      const int64_t row0 = static_cast<int64_t>(seq.q0 + i0 + t * tile_tokens) * p.H + g * p.G;
      // where tile row x goes, in rows of the output
      auto out_row = [&](int x) {
        const int k = div_by_group(p, x);
        return row0 + static_cast<int64_t>(k) * p.H + (x - k * p.G);
      };
      // the whole row at once: one wait for tensor memory
      uint32_t o[D];
      if (zero) {
#pragma unroll
        for (int c = 0; c < D; ++c) o[c] = 0u;
      } else {
#pragma unroll
        for (int cb = 0; cb < D; cb += 32)
          tmem_ld32(tO + cb, *reinterpret_cast<uint32_t(*)[32]>(&o[cb]));
        tmem_ld_wait(o);
#pragma unroll
        for (int c = 0; c < D; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * inv_l);
      }
      if (p.out_f32) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<float*>(p.O) +
                                              out_row(in_use ? r : quarter * 32) * D);
        if (in_use) {
#pragma unroll
          for (int c = 0; c < D / 4; ++c)
            dst[c] = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
        }
      } else {
        // bf16 rows go through this warp's part of the tile's Q block, which
        // its products have read, so that a store writes whole rows: 16-byte
        // piece c of row x at place c ^ (x & 7)
        constexpr int kPieces = D / 8;
        uint4* stg = reinterpret_cast<uint4*>(gbase + C::kOffQ + t * C::kQTileBytes) +
                     quarter * 32 * kPieces;
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
          uint4 v;
          v.x = pack_bf16x2(__uint_as_float(o[8 * c + 0]), __uint_as_float(o[8 * c + 1]));
          v.y = pack_bf16x2(__uint_as_float(o[8 * c + 2]), __uint_as_float(o[8 * c + 3]));
          v.z = pack_bf16x2(__uint_as_float(o[8 * c + 4]), __uint_as_float(o[8 * c + 5]));
          v.w = pack_bf16x2(__uint_as_float(o[8 * c + 6]), __uint_as_float(o[8 * c + 7]));
          stg[lane * kPieces + (c ^ (lane & 7))] = v;
        }
        __syncwarp();
        const int piece = lane % kPieces;
#pragma unroll 4
        for (int x = lane / kPieces; x < rows_here; x += 32 / kPieces) {
          const uint4 v = stg[x * kPieces + (piece ^ (x & 7))];
          reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.O) +
                                   out_row(quarter * 32 + x) * D)[piece] = v;
        }
      }
    }
  }

  if (p.splits > 1) {
    // ---- merge the splits: every CTA of the cluster takes a share of the
    // rows, fetches their m and l from all splits, works out the weights, and
    // sums up the outputs four columns at a time.
    __syncwarp();
    cluster_sync();  // every split's m, l, O and bad-page flag are in its shared memory
    const int S = p.splits;
    const int tile_rows = tile_tokens * p.G;  // those of a full tile
    const int rows = min(block_tokens, max(0, seq.n - i0)) * p.G;
    auto smem_row = [&](int row) { return row < tile_rows ? row : row + kBlockM - tile_rows; };
    const int per = (rows + S - 1) / S;
    const int r0 = split * per;
    const int mine = max(0, min(rows, r0 + per) - r0);
    float* weights = reinterpret_cast<float*>(gbase + C::kOffW);  // [row of mine][S]
    const uint32_t xo_s = base, xm_s = base + C::kOffM;
    float* lm = weights + C::kShare;
    float* ll = lm + C::kShare;
    const bool bad = any_bad(smem_u32(const_cast<int*>(bad_page)), S);
#pragma unroll 1
    for (int x = threadIdx.x; x < mine * S; x += C::kThreads) {
      const int k = x / S;
      const uint32_t s = x - k * S, row = smem_row(r0 + k);
      lm[x] = ld_cluster_f32(cluster_map(xm_s + 4u * row, s));
      ll[x] = ld_cluster_f32(cluster_map(xm_s + 4u * (NQT * kBlockM + row), s));
    }
    __syncthreads();
#pragma unroll 1
    for (int x = threadIdx.x; x < mine * S; x += C::kThreads) {
      const int k = x / S;
      weights[x] = bad ? 0.f : split_weight(lm + k * S, ll + k * S, 1, S, x - k * S);
    }
    __syncthreads();
    const int total = mine * (D / 4);
    // place e of this CTA's share: its shared address, its output element
    auto place_from = [&](int row, int c) {
      return xo_s + 4u * (smem_row(r0 + row) * C::kXRow + c);
    };
    auto place_to = [&](int row, int c) {
      const int i = div_by_group(p, r0 + row);
      return (static_cast<int64_t>(seq.q0 + i0 + i) * p.H + g * p.G + (r0 + row - i * p.G)) * D + c;
    };
    if (total < 4 * C::kThreads) {
      // few places: several threads to one where there are threads to spare
      const int sharers = merge_sharers(total, S, C::kThreads);
#pragma unroll 1
      for (int f0 = 0; f0 < total; f0 += C::kThreads / sharers) {
        const int e = f0 + static_cast<int>(threadIdx.x) / sharers;
        const int row = e / (D / 4), c = e % (D / 4) * 4;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (e < total) {
          const uint32_t from = place_from(row, c);
#pragma unroll 4
          for (int s = threadIdx.x % sharers; s < S; s += sharers)
            add_split(o, from, s, weights[row * S + s]);
        }
        sum_sharers(o, sharers);
        if (e < total && threadIdx.x % sharers == 0) store_out4(p, place_to(row, c), o);
      }
    } else {
      // many: eight places of a thread at a time, a remote load each under way
      constexpr int N = 8;
#pragma unroll 1
      for (int f0 = threadIdx.x; f0 < total; f0 += N * C::kThreads) {
        float4 o[N];
#pragma unroll
        for (int k = 0; k < N; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int s = 0; s < S; ++s) {
          float4 v[N];
          const uint32_t there = cluster_map(xo_s, static_cast<uint32_t>(s));
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const int e = min(f0 + k * C::kThreads, total - 1);
            v[k] = ld_cluster_f32x4(there + (place_from(e / (D / 4), e % (D / 4) * 4) - xo_s));
          }
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const int e = min(f0 + k * C::kThreads, total - 1);
            const float w = weights[e / (D / 4) * S + s];
            if (w != 0.f) {  // as in add_split
              o[k].x = fmaf(w, v[k].x, o[k].x);
              o[k].y = fmaf(w, v[k].y, o[k].y);
              o[k].z = fmaf(w, v[k].z, o[k].z);
              o[k].w = fmaf(w, v[k].w, o[k].w);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const int e = f0 + k * C::kThreads;
          if (e < total) store_out4(p, place_to(e / (D / 4), e % (D / 4) * 4), o[k]);
        }
      }
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while another still reads its shared memory
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::kMmaWarp) tmem_dealloc<C::kTmemCols>(tmem);
}

// Blocks that T packed tokens of B sequences, max_new each, can make, for
// every kv head: a block per block_tokens tokens and a partial one per
// sequence, and no more than each sequence can have.
int64_t block_bound(const PagedSdpaArgs& a, int block_tokens) {
  const int64_t seqs = a.T < a.pages.B ? a.T : a.pages.B;
  const int64_t each = (a.max_new + block_tokens - 1) / block_tokens;
  const int64_t packed = a.T / block_tokens + seqs;
  return (seqs * each < packed ? seqs * each : packed) * a.pages.kv_heads;
}

template <int D, int NQT, int NST, int BN>
cudaError_t launch_impl(PagedSdpaArgs a, const DeviceCtl& ctl) {
  using C = RowsCfg<D, NQT, NST, BN>;
  CUtensorMap q, k, v;
  if (!paged_tensor_maps(a, D, kBlockM / a.G, BN, &q, &k, &v)) return cudaErrorInvalidValue;
  const int64_t blocks = block_bound(a, NQT * (kBlockM / a.G));
  if (a.splits == 0)
    a.splits = paged_default_splits(
        blocks, static_cast<int64_t>(a.pages.cols) << a.pages.page_shift, C::kThreads, C::kSmemBytes);
  if (blocks * a.splits > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  auto kern = sdpa_paged_rows_kernel<D, NQT, NST, BN>;
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
  e = cudaLaunchKernelEx(&cfg, kern, q, k, v, paged_params(a, ctl));
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_sdpa_paged_rows(const PagedSdpaArgs& a, const DeviceCtl& ctl) {
  // Two query tiles per CTA halve the key/value traffic per row and keep the
  // tensor core busy during one tile's softmax: taken when a sequence can
  // have two tiles of new tokens.
  const bool two = a.max_new > kBlockM / a.G;
  if (a.pages.d == 64)
    return two ? launch_impl<64, 2, 3, 64>(a, ctl) : launch_impl<64, 1, 2, 128>(a, ctl);
  return two ? launch_impl<128, 2, 2, 128>(a, ctl) : launch_impl<128, 1, 2, 64>(a, ctl);
}

}  // namespace mha
