// sdpa_paged_rows.cuh -- what the query-tile forms of the paged attention share
// around their key loops: which block of tokens a CTA takes, the output of a
// tile, and the merge of a cluster's splits.
#pragma once

#include "sdpa_paged.cuh"

namespace mha {

constexpr int kRowsM = 128;      // query rows per tile = TMEM lanes
constexpr int kMaxSorted = 256;  // sequences that a CTA ranks by length

// A CTA's block: sequence b (-1: none), kv head g, and the block's first token
// of the sequence.
struct RowsBlock {
  int b, g, i0;
  PagedSeq seq;
};

// Which (sequence, kv head, block of tokens) this CTA computes: blocks
// are numbered sequence by sequence, longest first (CTAs start in grid
// order, so long ones do not trail alone at the end; up to kMaxSorted
// sequences, ranked by every CTA itself); in a sequence head by head (a
// head's blocks run at about the same time and share its pages in L2), in a
// head from the last tokens to the first, which see fewer keys.
// The whole CTA calls this; barriers and tensor memory that were set up before
// are visible to it afterwards.  `scratch`: shared memory, 4 * (3 *
// kMaxSorted + 1) bytes, that the copies to follow may write over; pick: three
// integers.
template <int kThreads>
__device__ __forceinline__ RowsBlock rows_block(const PagedParams& p, uint8_t* scratch,
                                                volatile int* pick, int block_tokens) {
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  int* lens_s = reinterpret_cast<int*>(scratch);
  int* off_s = lens_s + kMaxSorted;
  int* order_s = off_s + kMaxSorted + 1;
  const bool sorted = p.B > 1 && p.B <= kMaxSorted;
  if (sorted) {
    for (int i = threadIdx.x; i <= p.B; i += kThreads) {
      off_s[i] = paged_offset(p, i);
      if (i < p.B) lens_s[i] = __ldg(p.kv_len + i);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.B; c += kThreads) {
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
  RowsBlock k{};
  k.b = pick[0];
  k.g = pick[1];
  k.i0 = pick[2] * block_tokens;
  if (k.b >= 0) k.seq = seq_of(k.b);
  if (sorted) {
    fence_proxy_async_smem();  // the copies that follow write over the sequences
    __syncthreads();
  }
  return k;
}

// One warp's 32 rows of a tile's output: O in tensor memory at tO times inv_l,
// or zeros.  row0: the row of the output of the tile's first token and head;
// stage: this tile's Q block in shared memory, which its products have read.
template <int D>
__device__ __forceinline__ void rows_store(const PagedParams& p, uint32_t tO, bool zero,
                                           float inv_l, int quarter, int tile_rows, int64_t row0,
                                           uint8_t* stage) {
  const int lane = threadIdx.x & 31;
  const int rows_here = min(32, tile_rows - quarter * 32);
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
                                          out_row(quarter * 32 + (lane < rows_here ? lane : 0)) * D);
    if (lane < rows_here) {
#pragma unroll
      for (int c = 0; c < D / 4; ++c)
        dst[c] = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
    }
  } else {
    // bf16 rows go through this warp's part of the tile's Q block, which
    // its products have read, so that a store writes whole rows: 16-byte
    // piece c of row x at place c ^ (x & 7)
    constexpr int kPieces = D / 8;
    uint4* stg = reinterpret_cast<uint4*>(stage) +
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

// Merge the splits: every CTA of the cluster takes a share of the rows, fetches
// their m and l from all splits, works out the weights, and sums up the outputs
// four columns at a time.  Between cluster barriers; xo_s, xm_s: shared
// addresses of the partial outputs [NQT * 128][D + 4] and of m and l of every
// row; w_at: three times kShare floats.  The block's first kThreads threads
// (whole warps) call this.
template <int D, int NQT, int kThreads>
__device__ __forceinline__ void rows_merge(const PagedParams& p, const PagedSeq& seq, int g, int i0,
                                           int split, int tile_tokens, uint32_t xo_s,
                                           uint32_t xm_s, float* w_at, volatile int* bad_page) {
  constexpr int kShare = NQT * kRowsM + kPagedMaxSplits;
  const int block_tokens = NQT * tile_tokens;
  const int S = p.splits;
  const int tile_rows = tile_tokens * p.G;  // those of a full tile
  const int rows = min(block_tokens, max(0, seq.n - i0)) * p.G;
  auto smem_row = [&](int row) { return row < tile_rows ? row : row + kRowsM - tile_rows; };
  const int per = (rows + S - 1) / S;
  const int r0 = split * per;
  const int mine = max(0, min(rows, r0 + per) - r0);
  float* weights = w_at;  // [row of mine][S]
  float* lm = weights + kShare;
  float* ll = lm + kShare;
  const bool bad = any_bad(smem_u32(const_cast<int*>(bad_page)), S);
#pragma unroll 1
  for (int x = threadIdx.x; x < mine * S; x += kThreads) {
    const int k = x / S;
    const uint32_t s = x - k * S, row = smem_row(r0 + k);
    lm[x] = ld_cluster_f32(cluster_map(xm_s + 4u * row, s));
    ll[x] = ld_cluster_f32(cluster_map(xm_s + 4u * (NQT * kRowsM + row), s));
  }
  asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
#pragma unroll 1
  for (int x = threadIdx.x; x < mine * S; x += kThreads) {
    const int k = x / S;
    weights[x] = bad ? 0.f : split_weight(lm + k * S, ll + k * S, 1, S, x - k * S);
  }
  asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
  const int total = mine * (D / 4);
  // place e of this CTA's share: its shared address, its output element
  auto place_from = [&](int row, int c) {
    return xo_s + 4u * (smem_row(r0 + row) * (D + 4) + c);
  };
  auto place_to = [&](int row, int c) {
    const int i = div_by_group(p, r0 + row);
    return (static_cast<int64_t>(seq.q0 + i0 + i) * p.H + g * p.G + (r0 + row - i * p.G)) * D + c;
  };
  if (total < 4 * kThreads) {
    // few places: several threads to one where there are threads to spare
    const int sharers = merge_sharers(total, S, kThreads);
#pragma unroll 1
    for (int f0 = 0; f0 < total; f0 += kThreads / sharers) {
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
    for (int f0 = threadIdx.x; f0 < total; f0 += N * kThreads) {
      float4 o[N];
#pragma unroll
      for (int k = 0; k < N; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int s = 0; s < S; ++s) {
        float4 v[N];
        const uint32_t there = cluster_map(xo_s, static_cast<uint32_t>(s));
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const int e = min(f0 + k * kThreads, total - 1);
          v[k] = ld_cluster_f32x4(there + (place_from(e / (D / 4), e % (D / 4) * 4) - xo_s));
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const int e = min(f0 + k * kThreads, total - 1);
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
        const int e = f0 + k * kThreads;
        if (e < total) store_out4(p, place_to(e / (D / 4), e % (D / 4) * 4), o[k]);
      }
    }
  }
}

// Blocks that T packed tokens of B sequences, max_new each, can make, for
// every kv head: a block per block_tokens tokens and a partial one per
// sequence, and no more than each sequence can have.
inline int64_t rows_block_bound(const PagedSdpaArgs& a, int block_tokens) {
  const int64_t seqs = a.T < a.pages.B ? a.T : a.pages.B;
  const int64_t each = (a.max_new + block_tokens - 1) / block_tokens;
  const int64_t packed = a.T / block_tokens + seqs;
  return (seqs * each < packed ? seqs * each : packed) * a.pages.kv_heads;
}

}  // namespace mha
