/*
 * mha.h -- C ABI of the GB300 (sm_103a) multi-head scaled dot-product
 * attention library (libmha_gb300.so).
 *
 * What the library computes
 *   Attention(Q, K, V) = softmax(Q K^T * scale + M) V  per (batch, head),
 *   with scale = 1/sqrt(d_k) by default and M an additive 0/-inf mask
 *     -- "How Transformers Work" (worksonmygpu.com), "Scaled dot-product
 *        attention"; "The Transformer" (hoshank.vercel.app), "The
 *        Mathematics"; masks: "The Transformer" (rayaq.ca), "Masks: who may
 *        look at whom".
 *   MultiHead(x_q, x_kv) = Concat(head_1..head_h) W^O,
 *   head_i = Attention(x_q W^Q_i, x_kv W^K_i, x_kv W^V_i)
 *     -- hoshank.vercel.app, "The Mathematics" (multi-head equation);
 *        "32 Transformer" (ml-canon-en), "PyTorch Implementation": y = x @ W,
 *        head i = column block i of the projection, heads concatenated in
 *        order before W^O.  No bias terms.
 *
 * Conventions shared by every entry point
 *   - Tensors are dense, row-major (C order), in device memory unless stated
 *     otherwise, and owned by the caller.  Every tensor pointer must be
 *     16-byte aligned (TMA requirement); pointers to distinct tensors must
 *     not overlap, except x_kv == x_q (self-attention).
 *   - Element type: MHA_BF16 = bfloat16 (uint16 bit pattern), MHA_F32 = IEEE
 *     float.  bf16 work accumulates in fp32.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy
 *     default stream).  Arguments are validated on the host before anything
 *     is launched; a call that returns an error has launched nothing.
 *   - Errors are returned, never printed; the library never aborts.
 *   - Device-side conditions (a key length outside [1, Lk], a pipeline wait
 *     that exceeded its time limit) set a per-device error word that
 *     mha_check() reads.  The affected rows are written as zeros.
 *   - Paged key/value caches are described by an mha_kv_pages (below);
 *     its pools follow the same alignment rule, its page table and lengths
 *     are 4-byte aligned device int32 arrays.
 *   - Masks: mask_kind is a bit set of MHA_MASK_CAUSAL (key j blocked for
 *     query i when j > i; requires Lq == Lk) and MHA_MASK_KEY_PADDING (key j
 *     blocked for batch item b when j >= key_lengths[b]).  There are no
 *     boolean mask tensors, so no mask polarity to get wrong.
 */
#ifndef GB300_MHA_H
#define GB300_MHA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MHA_OK = 0,
    MHA_ERR_INVALID_ARG = 1, /* null/misaligned pointer, bad size, bad mask */
    MHA_ERR_UNSUPPORTED = 2, /* valid request outside what is implemented */
    MHA_ERR_CUDA = 3,        /* a CUDA runtime/driver call failed */
    MHA_ERR_OOM = 4,         /* device allocation failed (mha_create) */
    MHA_ERR_TIMEOUT = 5,     /* a kernel pipeline wait gave up (mha_check) */
    MHA_ERR_DEVICE = 6       /* device-side argument error, e.g. a key
                                length outside [1, Lk] (mha_check) */
} mha_status;

typedef enum {
    MHA_F32 = 0,
    MHA_BF16 = 1,
    MHA_E4M3 = 2 /* 8 bits, sign, 4 of exponent (bias 7), 3 of mantissa, largest
                    448, no infinities; the paged cache's _e4m3 calls, the
                    calls on selected pages and kv_pages_bounds only */
} mha_dtype;

enum {
    MHA_MASK_NONE = 0,
    MHA_MASK_CAUSAL = 1,
    MHA_MASK_KEY_PADDING = 2,
    /* sdpa_decode and sdpa_paged only: query i of the newest Lq sees keys
     * j <= len_b - Lq + i */
    MHA_MASK_CAUSAL_BOTTOM_RIGHT = 4
};

/* Largest number of new queries per (batch item, head) sdpa_decode takes. */
#define MHA_DECODE_MAX_QUERIES 16

/* Same type as cudaStream_t, declared here so the header needs no CUDA
 * include. */
typedef struct CUstream_st *mha_stream;

/* Opaque layer handle: owns the Q/K/V/context workspace for one d_model and
 * element type. */
typedef struct mha_ctx *mha_handle;

/*
 * sdpa_forward -- scaled dot-product attention for B*H independent heads.
 *   Q [B, H, Lq, d], K [B, H, Lk, d], V [B, H, Lk, d]  (in_dtype)
 *   O [B, H, Lq, d]                                    (out_dtype)
 *   scale       : multiplier of Q K^T; 0 selects 1/sqrt(d); must be finite
 *                 and >= 0.
 *   mask_kind   : bit set of MHA_MASK_*; CAUSAL requires Lq == Lk.
 *   key_lengths : device int32[B], required iff KEY_PADDING is set; each
 *                 value must lie in [1, Lk] (checked on the device).
 * Supported: in_dtype BF16 with d in {64, 128} (tcgen05 tensor-core path,
 * out_dtype BF16 or F32); in_dtype F32 with 1 <= d <= 128 (fp32 CUDA-core
 * path, out_dtype F32).  B, H, Lq may be 0 (nothing is launched); Lk >= 1.
 * Returns MHA_OK, MHA_ERR_INVALID_ARG, MHA_ERR_UNSUPPORTED or MHA_ERR_CUDA.
 */
mha_status sdpa_forward(const void *Q, const void *K, const void *V, void *O,
                        int B, int H, int Lq, int Lk, int d, float scale,
                        int mask_kind, const int32_t *key_lengths,
                        mha_dtype in_dtype, mha_dtype out_dtype,
                        mha_stream stream);

/*
 * sdpa_forward_host -- sdpa_forward on host buffers: Q, K, V (and the key
 * lengths) are copied in, attended and O is copied out, in about sixteen
 * chunks of (b, h) heads whose copies overlap the attention of other chunks
 * (every head is independent: "How Transformers Work" (worksonmygpu.com),
 * "Multi-head attention").
 *   Qh, Kh, Vh, Oh : host, same shapes and types as sdpa_forward; pinned
 *             (page-locked) memory lets the copies run asynchronously.
 *   key_lengths_h : host int32[B] or NULL, as sdpa_forward's key_lengths.
 *   workspace : device, 256-byte aligned, at least
 *             sdpa_forward_host_workspace_bytes(...) bytes; the call keeps
 *             device copies of Q, K, V, O and the lengths there.
 *   stream    : the call is ordered after work already queued on `stream`,
 *             and `stream` covers it: Oh is complete once `stream` has been
 *             synchronised.  Two internal copy streams and a second compute
 *             stream carry the overlap.
 * Same dtypes, head sizes and checks as sdpa_forward.  The call allocates
 * nothing on the device; it creates its internal streams and events once per
 * device.  Calls on one device are serialised on the host while they
 * enqueue.
 * Returns MHA_OK, MHA_ERR_INVALID_ARG, MHA_ERR_UNSUPPORTED or MHA_ERR_CUDA.
 */
mha_status sdpa_forward_host(const void *Qh, const void *Kh, const void *Vh, void *Oh,
                             int B, int H, int Lq, int Lk, int d, float scale,
                             int mask_kind, const int32_t *key_lengths_h,
                             mha_dtype in_dtype, mha_dtype out_dtype,
                             void *workspace, size_t workspace_bytes, mha_stream stream);

/* Device workspace sdpa_forward_host needs, in bytes (0 for bad arguments). */
size_t sdpa_forward_host_workspace_bytes(int B, int H, int Lq, int Lk, int d,
                                         mha_dtype in_dtype, mha_dtype out_dtype);

/*
 * sdpa_forward_float_mask -- sdpa_forward with an additive float mask added
 * to the scaled scores, the optional mask of the reference SDPA that "The
 * Transformer" (rayaq.ca) describes in "Attention, by hand" (with -inf
 * giving weight exactly 0, "Masks: who may look at whom").
 *   add_mask : device float32; element (b, h, i, j) at
 *              add_mask[b*mask_stride_b + h*mask_stride_h + i*Lk + j]
 *              (strides in elements, >= 0; 0 broadcasts over that axis;
 *              rows of Lk contiguous values).  Entries must be finite or
 *              -inf.  4-byte aligned.
 *   Other arguments, layouts and support as for sdpa_forward; mask_kind and
 *   key_lengths still apply on top.  A query row whose keys are all blocked
 *   has no defined softmax and is written as zeros.
 * Returns MHA_OK, MHA_ERR_INVALID_ARG, MHA_ERR_UNSUPPORTED or MHA_ERR_CUDA.
 */
mha_status sdpa_forward_float_mask(const void *Q, const void *K, const void *V,
                                   void *O, int B, int H, int Lq, int Lk,
                                   int d, float scale, int mask_kind,
                                   const int32_t *key_lengths,
                                   const float *add_mask,
                                   int64_t mask_stride_b,
                                   int64_t mask_stride_h, mha_dtype in_dtype,
                                   mha_dtype out_dtype, mha_stream stream);

/*
 * sdpa_decode -- attention of Lq <= 16 new queries per (batch item, head)
 * against a key/value cache: the decoder's masked self-attention while it
 * generates left to right, reusing the keys and values it has stored ("How
 * Transformers Work" (worksonmygpu.com), "What changed since 2017"; "The
 * Transformer" (hoshank.vercel.app), "The Breakthrough"; "The Transformer"
 * (rayaq.ca), "The decoder stack").
 *   Q       [B, H, Lq, d] bf16: the queries of the newest Lq positions.
 *   K_cache [B, H, Lk, d] bf16, V_cache [B, H, Lk, d] bf16: a cache of
 *           capacity Lk; batch item b holds len_b tokens in rows
 *           [0, len_b), the newest Lq of them being the queries' own.
 *   O       [B, H, Lq, d], out_dtype BF16 or F32.
 *   scale   : as for sdpa_forward (0 selects 1/sqrt(d)).
 *   mask_kind : bit set of MHA_MASK_KEY_PADDING (len_b = kv_lengths[b]; else
 *           every item holds Lk tokens) and MHA_MASK_CAUSAL_BOTTOM_RIGHT
 *           (query i sees keys j <= len_b - Lq + i; without it every query
 *           sees all len_b keys, as cross-attention to an encoder memory).
 *           MHA_MASK_CAUSAL is not accepted here.
 *   kv_lengths : device int32[B], given iff KEY_PADDING is set; each value
 *           must lie in [1, Lk], and in [Lq, Lk] with the causal bit
 *           (checked on the device: MHA_ERR_DEVICE from mha_check, rows
 *           written as zeros).
 *   num_splits : CTAs that share one (b, h)'s keys, 1..16, merged exactly
 *           through one thread-block cluster; 0 picks a default
 *           (sdpa_decode_splits).
 * d must be 64 or 128; Q, K_cache, V_cache and O 16-byte aligned.  B or H
 * may be 0 (nothing is launched).  The call allocates nothing.
 * Returns MHA_OK, MHA_ERR_INVALID_ARG, MHA_ERR_UNSUPPORTED (Lq > 16, other
 * d) or MHA_ERR_CUDA.
 */
mha_status sdpa_decode(const void *Q, const void *K_cache, const void *V_cache,
                       void *O, int B, int H, int Lq, int Lk, int d,
                       float scale, int mask_kind, const int32_t *kv_lengths,
                       mha_dtype out_dtype, int num_splits,
                       mha_stream stream);

/* The split count sdpa_decode uses for num_splits = 0 (0 for bad sizes). */
int sdpa_decode_splits(int B, int H, int Lk, int d);

/*
 * sdpa_forward_lse -- sdpa_forward (bf16 inputs) that also writes, per query
 * row, the base-2 log-sum-exp of the scaled scores, which the backward pass
 * needs to recompute the attention weights:
 *   lse[b, h, i] = log2( sum_j 2^((scale * <Q_i, K_j> + M_ij) * log2(e)) )
 * (+inf for a row with no visible key).
 *   lse : device fp32 [B, H, Lq], 4-byte aligned, caller-owned.
 * Other arguments, layouts, support and errors as for sdpa_forward with
 * in_dtype = MHA_BF16.
 */
mha_status sdpa_forward_lse(const void *Q, const void *K, const void *V, void *O,
                            float *lse, int B, int H, int Lq, int Lk, int d,
                            float scale, int mask_kind,
                            const int32_t *key_lengths, mha_dtype out_dtype,
                            mha_stream stream);

/* Workspace sdpa_backward needs, in bytes (one fp32 per query row). */
size_t sdpa_backward_workspace_bytes(int B, int H, int Lq);

/*
 * sdpa_backward -- gradients of scaled dot-product attention (the training
 * step through the attention formula of "How Transformers Work"
 * (worksonmygpu.com), "Scaled dot-product attention"): given dO = dL/dO for
 * O = sdpa_forward(Q, K, V),
 *   dV = P^T dO,  dS = P * (dO V^T - rowsum(dO * O)),
 *   dQ = scale * dS K,  dK = scale * dS^T Q.
 *   Q, O, dO [B, H, Lq, d] bf16; K, V [B, H, Lk, d] bf16 (as in the forward).
 *   lse     : fp32 [B, H, Lq] from sdpa_forward_lse on the same inputs.
 *   dQ      : fp32 [B, H, Lq, d], written once (its sum over keys stays on
 *             the chip; nothing is accumulated in global memory).
 *   dK, dV  : [B, H, Lk, d] of grad_dtype (MHA_BF16 or MHA_F32).
 *   scale, mask_kind, key_lengths : as in the forward (CAUSAL and
 *             KEY_PADDING; no float mask).
 *   workspace : device, >= sdpa_backward_workspace_bytes(B, H, Lq) bytes.
 * d must be 64 or 128; all pointers 16-byte aligned.  Blocked keys receive
 * zero gradient; a query row with no visible key gets dQ = 0.  The call
 * allocates nothing.  Two kernels run on `stream`: dK and dV (a CTA per key
 * tile) and dQ (a CTA per query tile), after the row dot products D.
 * Returns MHA_OK, MHA_ERR_INVALID_ARG, MHA_ERR_UNSUPPORTED or MHA_ERR_CUDA.
 */
mha_status sdpa_backward(const void *Q, const void *K, const void *V,
                         const void *O, const void *dO, const float *lse,
                         float *dQ, void *dK, void *dV, int B, int H, int Lq,
                         int Lk, int d, float scale, int mask_kind,
                         const int32_t *key_lengths, mha_dtype grad_dtype,
                         void *workspace, size_t workspace_bytes,
                         mha_stream stream);

/*
 * sinusoidal_pe -- the positional-encoding table, fp32 [n_pos, d_model]:
 * row r holds PE(first_pos + r, :) with PE(pos, 2i) = sin(pos / 10000^(2i/D))
 * and PE(pos, 2i+1) = cos(pos / 10000^(2i/D)) ("How Transformers Work"
 * (worksonmygpu.com), "Positional encoding"; "The Transformer"
 * (hoshank.vercel.app), "The Mathematics").  Each value is the fp64 sine or
 * cosine of the fp64 angle, rounded to fp32.  pe: device, 4-byte aligned,
 * caller-owned.  Built once per length and reused.
 * Returns MHA_OK, MHA_ERR_INVALID_ARG or MHA_ERR_CUDA.
 */
mha_status sinusoidal_pe(float *pe, int first_pos, int n_pos, int d_model,
                         mha_stream stream);

/*
 * embed_pe_forward -- the first layer's input in one pass:
 *   x[b, l, :] = table[ids[b, l], :] * scale + pe[pos_offset + l, :]
 * the token embedding scaled by sqrt(d_model) plus the positional encoding
 * ("The Transformer" (rayaq.ca), "Embeddings and positions" and the encode
 * step of "Implementation").
 *   ids   : device int32 [B, L]; each must lie in [0, vocab) (checked on the
 *           device: MHA_ERR_DEVICE from mha_check, the row written as zeros).
 *   table : device [vocab, d_model] of dtype (BF16 or F32), 16-byte aligned.
 *   pe    : device fp32 [pe_rows, d_model] from sinusoidal_pe (first_pos 0),
 *           16-byte aligned; pos_offset + L <= pe_rows.
 *   x     : device [B, L, d_model] of dtype, 16-byte aligned; the sum is
 *           taken in fp32 and rounded once.
 *   scale : 0 selects sqrt(d_model); otherwise finite and >= 0.
 * Returns MHA_OK, MHA_ERR_INVALID_ARG or MHA_ERR_CUDA.
 */
mha_status embed_pe_forward(const int32_t *ids, const void *table, int vocab,
                            const float *pe, int pe_rows, void *x, int B,
                            int L, int d_model, int pos_offset, float scale,
                            mha_dtype dtype, mha_stream stream);

/*
 * A paged key/value cache: the rows of a sequence's keys and values lie in
 * pages of page_size rows that need not be neighbours, so that no sequence
 * reserves rows it does not hold and sequences can share pages (the
 * PagedAttention remark of "How Transformers Work" (worksonmygpu.com), "What
 * changed since 2017").  One page table serves `layers` pools.
 *   K, V : pools.  Row s of page p, kv head g, layer y starts at element
 *          y*layer_stride + p*page_stride + (g*page_size + s)*d.
 *   page_stride  : 0 selects the dense kv_heads*page_size*d.
 *   layer_stride : 0 selects num_pages*page_stride.  Both are multiples of d
 *          and at least one page.
 *   page_table : device int32 [B, table_cols]; token j of sequence b lies in
 *          row j % page_size of page page_table[b][j / page_size].  Entries
 *          behind a sequence's last held page are never read.
 *   kv_lengths : device int32 [B], tokens held by each sequence.
 *   B : sequences; with none, page_table and kv_lengths may be NULL.
 * page_size is a power of two from 16 to 256; table_cols*page_size <= 2^30.
 */
typedef struct {
    void *K, *V;
    mha_dtype dtype;
    int num_pages, page_size, kv_heads, d, layers;
    int64_t page_stride, layer_stride;
    int32_t *page_table;
    int32_t *kv_lengths;
    int B, table_cols;
} mha_kv_pages;

/*
 * A paged cache in 8 bits: pools of MHA_E4M3 codes and, for every page and kv
 * head, one scale for its keys and one for its values; row = code * scale.
 *   K, V : device fp32 [layers, num_pages, kv_heads], dense, 4-byte aligned.
 *          A scale is finite and >= 0; those of pages that no sequence holds
 *          may be anything.
 * The calls that take an mha_kv_scales expect pages->dtype MHA_E4M3; d is a
 * multiple of 16.  Strides count elements, bytes here.
 */
typedef struct {
    float *K, *V;
} mha_kv_scales;

/*
 * sdpa_paged -- attention of each sequence's newest tokens over its paged
 * cache: one token each while decoding, a few, or a long chunk of a prompt,
 * mixed in one call.  Query heads may share key/value heads.
 *   Q : bf16, T packed tokens; head h of token t at t*q_token_stride + h*d
 *       (0 selects the dense H*d).  q_token_stride is a multiple of d.
 *   q_offsets : device int32 [B+1]; sequence b's queries are the tokens
 *       [q_offsets[b], q_offsets[b+1]), the newest n_b of the kv_lengths[b]
 *       tokens its pages hold (their own keys and values among them).  A
 *       sequence without queries is passed over.
 *   O : [T, H, d] (the concatenated heads), out_dtype BF16 or F32.  Rows of
 *       tokens that belong to no sequence are left as they were.
 *   H : a multiple of kv_heads; head h reads kv head h / (H / kv_heads), and
 *       H / kv_heads <= 128.
 *   max_new : the largest n_b, 1 <= max_new (0 will do for T = 0).  Up to 16
 *       rows (max_new times the query heads of a kv head) take a kernel of
 *       their own, so a tight bound matters while decoding; one kernel serves
 *       all sequences of a call.
 *   scale : as for sdpa_forward (0 selects 1/sqrt(d)).
 *   mask_kind : MHA_MASK_CAUSAL_BOTTOM_RIGHT (query i of n_b sees the tokens
 *       j <= kv_lengths[b] - n_b + i) or MHA_MASK_NONE (it sees all).
 *   num_splits : CTAs that share one block's keys, 1..16, merged exactly
 *       through one thread-block cluster; 0 picks a default.
 * The cache is pages->dtype BF16 with d in {64, 128}; `layer` picks the pool.
 * Scores, exponentials and sums are fp32.  The weights are rounded to bf16
 * before they meet V, as sdpa_forward's are, whatever out_dtype: an output
 * moves by up to 2^-8 sum_j w_j |v_j|, beside its own rounding.
 * Rows of a page that lie behind the sequence's length may hold anything.
 * The keys and values that a sequence holds must be finite, those of new
 * tokens that a query does not see among them.  A NaN in a query reaches that
 * query's row alone.
 * Checked on the device (MHA_ERR_DEVICE from mha_check): kv_lengths[b] in
 * [max(1, n_b), table_cols*page_size] (from 1 without the causal bit) and
 * page numbers in [0, num_pages) -- every row that would read through the bad
 * entry is written as zeros, and other rows of that sequence may be;
 * q_offsets ascending in [0, T] and n_b <= max_new -- nothing is written for
 * such a sequence.  Where offsets descend, ranges overlap: rows of the other
 * sequences may be left unwritten too, or hold either one's result.
 * T or B may be 0.  The call allocates nothing and needs no workspace.
 * Returns MHA_OK, MHA_ERR_INVALID_ARG, MHA_ERR_UNSUPPORTED or MHA_ERR_CUDA.
 */
mha_status sdpa_paged(const void *Q, int64_t q_token_stride,
                      const mha_kv_pages *pages, int layer,
                      const int32_t *q_offsets, void *O, int T, int H,
                      int max_new, float scale, int mask_kind,
                      mha_dtype out_dtype, int num_splits, mha_stream stream);

/*
 * sdpa_paged_e4m3 -- sdpa_paged over a cache in 8 bits.  Q is bf16; the rest is
 * as for sdpa_paged, but for the products' operands.  A query row meets the
 * keys' codes as two e4m3 parts, which together are off by at most 2^-17 of
 * the row's largest element (2^-21 with up to 16 rows, see max_new).  The
 * weights, times the values' scales, meet the values' codes as two e4m3 parts
 * (up to 16 rows: off by 2^-8 of a weight, or 2^-23 of the row's largest
 * product of weight and scale) or in fp16 (more rows: off by 2^-11 of a weight,
 * or 2^-31 of that product).  A key whose scale is 0 counts in that product
 * with 2^-30 of the others' (up to 16 rows) or 2^-60.  The value scales of one sequence, but for zeros, lie within 2^100 of each
 * other, 2^70 where some are 0.  An infinity in a query gives NaN in its row.
 * Half the bytes make single tokens over long caches up to twice as fast as
 * sdpa_paged; chunks of hundreds of new tokens and more, which the products and
 * the softmax bound, take up to a fifth longer.
 */
mha_status sdpa_paged_e4m3(const void *Q, int64_t q_token_stride,
                           const mha_kv_pages *pages,
                           const mha_kv_scales *scales, int layer,
                           const int32_t *q_offsets, void *O, int T, int H,
                           int max_new, float scale, int mask_kind,
                           mha_dtype out_dtype, int num_splits,
                           mha_stream stream);

/* How the rotation pairs a head's first rope_dim columns. */
enum {
    MHA_ROPE_INTERLEAVED = 0, /* (2i, 2i+1) */
    MHA_ROPE_HALF = 1         /* (i, i + rope_dim/2) */
};

/*
 * qk_norm_rope_forward -- the norm of every query and key head and the
 * rotation by its position, in one pass:
 *   z = x * rsqrt(mean(x^2) + eps) * gamma          over the d columns
 *   (y_a, y_b) = (z_a cos - z_b sin, z_b cos + z_a sin)
 * for the rope_dim/2 column pairs (a, b) of `pairing`; columns from rope_dim
 * on are z.  The rotation turns relative position into the dot product: the
 * shift-by-k property of the sinusoidal encoding ("How Transformers Work"
 * (worksonmygpu.com), "Positional encoding").
 *   Q : [B, L, H, d] with token stride q_token_stride (elements, 0 = H*d;
 *       e.g. a slice of one projection's output); K : likewise, Hkv heads.
 *   gamma_q, gamma_k : [d], of dtype.
 *   pe : fp32 [pe_rows, rope_dim] in sinusoidal_pe's layout: row p holds
 *        sin, cos of pair i at columns 2i, 2i+1 (sinusoidal_pe builds it
 *        for base 10000; any table of that layout will do).  16-byte aligned.
 *   positions : device int32 [B, L], each in [0, pe_rows) (checked on the
 *        device: MHA_ERR_DEVICE, the token's rows written as zeros), or NULL:
 *        token l is at pos_offset + l, and pos_offset + L <= pe_rows.
 *   Qo [B, H, L, d], Ko [B, Hkv, L, d] : of dtype.  With Hkv = H that is what
 *       sdpa_forward, sdpa_forward_lse and sdpa_backward take (the last two in
 *       BF16 alone); they know no shared key heads, so for Hkv < H the caller
 *       repeats Ko's heads, and sums dKo over the copies.
 *   eps : finite, > 0.
 * dtype BF16 or F32; the arithmetic is fp32, rounded once.  2 <= d <= 256,
 * rope_dim even in [2, d].  H or Hkv may be 0 (that part is skipped).
 * With d in {64, 128} and rope_dim a multiple of 16, Q, K (and their
 * strides) are read as 16-byte vectors; every pointer is 16-byte aligned and
 * token strides are multiples of 16 bytes there.
 * Returns MHA_OK, MHA_ERR_INVALID_ARG, MHA_ERR_UNSUPPORTED or MHA_ERR_CUDA.
 */
mha_status qk_norm_rope_forward(const void *Q, int64_t q_token_stride,
                                const void *K, int64_t k_token_stride,
                                const void *gamma_q, const void *gamma_k,
                                const float *pe, int pe_rows, int rope_dim,
                                int pairing, void *Qo, void *Ko, int B, int L,
                                int H, int Hkv, int d, int pos_offset,
                                const int32_t *positions, float eps,
                                mha_dtype dtype, mha_stream stream);

/*
 * qk_norm_rope_backward -- its gradient.  With dz the rotation of dQo by the
 * opposite angle, xh = x * rstd and u = dz * gamma:
 *   dQ = rstd * (u - xh * mean(u * xh)),   dgamma = sum over rows of dz * xh
 *   dQo [B, H, L, d] of dq_dtype, dKo [B, Hkv, L, d] of dk_dtype (BF16 or
 *       F32: sdpa_backward gives dQ in fp32).
 *   dQ, dK : of dtype, laid out as Q and K with token strides of their own.
 *   dgamma_q, dgamma_k : fp32 [d], overwritten; 16-byte aligned.
 *   workspace : device, 16-byte aligned, at least
 *       qk_norm_rope_backward_workspace_bytes(d) bytes; one call's at a time
 *       (captured graphs that may run at once need one each).
 * The sums run in a fixed order, in fp32 over a block's rows and fp64 over the
 * blocks: equal calls give equal bits.  A token with a
 * bad position gets zero rows and adds nothing to dgamma.
 * Other arguments, support and errors as for qk_norm_rope_forward.
 */
mha_status qk_norm_rope_backward(const void *Q, int64_t q_token_stride,
                                 const void *K, int64_t k_token_stride,
                                 const void *gamma_q, const void *gamma_k,
                                 const float *pe, int pe_rows, int rope_dim,
                                 int pairing, const void *dQo, const void *dKo,
                                 void *dQ, int64_t dq_token_stride, void *dK,
                                 int64_t dk_token_stride, float *dgamma_q,
                                 float *dgamma_k, int B, int L, int H, int Hkv,
                                 int d, int pos_offset,
                                 const int32_t *positions, float eps,
                                 mha_dtype dtype, mha_dtype dq_dtype,
                                 mha_dtype dk_dtype, void *workspace,
                                 size_t workspace_bytes, mha_stream stream);

/* Workspace qk_norm_rope_backward needs, in bytes (0 for a bad d). */
size_t qk_norm_rope_backward_workspace_bytes(int d);

/*
 * qk_norm_rope_paged -- the serving form: norm and rotation of T packed new
 * tokens, whose keys and values go straight into their pages.
 *   Q [T, H, d], K and V [T, kv_heads, d] : bf16, token strides as above.
 *   q_offsets, pages, layer : as for sdpa_paged, kv_lengths already counting
 *       the new tokens; token i of sequence b's n_b is at position
 *       kv_lengths[b] - n_b + i, which picks its row of pe and its page row.
 *   Qo : [T, H, d], ready for sdpa_paged.
 * Pages that receive rows must not be shared between sequences.  d is 64 or
 * 128, rope_dim a multiple of 16.
 * Checked on the device (MHA_ERR_DEVICE): kv_lengths[b] in [n_b,
 * table_cols*page_size], positions below pe_rows, page numbers -- such a
 * token's Qo rows are written as zeros and no page is touched for it; offsets
 * ascending in [0, T], where a token meets them -- nothing is written for it.
 * Tokens that belong to no sequence, ahead of the first or behind the last,
 * are passed over.
 * Returns MHA_OK, MHA_ERR_INVALID_ARG, MHA_ERR_UNSUPPORTED or MHA_ERR_CUDA.
 */
mha_status qk_norm_rope_paged(const void *Q, int64_t q_token_stride,
                              const void *K, int64_t k_token_stride,
                              const void *V, int64_t v_token_stride,
                              const void *gamma_q, const void *gamma_k,
                              const float *pe, int pe_rows, int rope_dim,
                              int pairing, void *Qo, const mha_kv_pages *pages,
                              int layer, const int32_t *q_offsets, int T,
                              int H, float eps, mha_stream stream);

/*
 * qk_norm_rope_paged_e4m3 -- qk_norm_rope_paged into a cache in 8 bits.  A page
 * keeps one scale per head, so the new rows of a page are stored together:
 *   need = the smallest power of two s >= 2^-100 with max |x| <= 448 s over
 *          the finite elements of the page's new rows; 0 where they are zeros
 *   s    = max(need, the page's scale), of a page without older rows need
 *   code = e4m3(x / s), to nearest, ties to even
 * and where s has grown, the older rows' codes become e4m3(code * old / s):
 * exact between powers of two, but for codes that leave the normal range
 * (x / s below 2^-6).  "Older" are the sequence's rows of that page ahead of
 * its new ones; what lies behind its length is not touched.  x is the normed,
 * rotated key or the value in fp32; elements that are not finite are stored
 * as NaN, and are NaN under a scale of 0, too.
 */
mha_status qk_norm_rope_paged_e4m3(
    const void *Q, int64_t q_token_stride, const void *K,
    int64_t k_token_stride, const void *V, int64_t v_token_stride,
    const void *gamma_q, const void *gamma_k, const float *pe, int pe_rows,
    int rope_dim, int pairing, void *Qo, const mha_kv_pages *pages,
    const mha_kv_scales *scales, int layer, const int32_t *q_offsets, int T,
    int H, float eps, mha_stream stream);

/*
 * kv_pages_fork -- n sequences continue n others (parallel samples, beams):
 * sequence children[i] takes parents[i]'s length and full pages (shared), and
 * the rows of its last, partly filled page are copied into page fresh[i], in
 * every layer.
 *   parents, children, fresh : device int32 [n].  fresh[i] must be held by no
 *       sequence; it is not read where the parent's last page is full.
 *       One parent may have many children.
 * The child's table entries behind its last page, and the rows of the fresh
 * page behind its length, are left as they were.
 * Checked on the device (MHA_ERR_DEVICE, that pair changes nothing): indexes
 * outside [0, B), a child that is also a parent of this call or named twice,
 * a needed fresh page outside [0, num_pages) or named twice, the parent's
 * length outside [0, table_cols*page_size], its last page's number.
 * Any dtype; d * element size must be a multiple of 16 bytes.
 * Returns MHA_OK, MHA_ERR_INVALID_ARG, MHA_ERR_UNSUPPORTED or MHA_ERR_CUDA.
 */
mha_status kv_pages_fork(const mha_kv_pages *pages, const int32_t *parents,
                         const int32_t *children, const int32_t *fresh, int n,
                         mha_stream stream);

/* kv_pages_fork_e4m3 -- kv_pages_fork of a cache in 8 bits: a fresh page takes
 * the scales of the page that it copies, in every layer. */
mha_status kv_pages_fork_e4m3(const mha_kv_pages *pages,
                              const mha_kv_scales *scales,
                              const int32_t *parents, const int32_t *children,
                              const int32_t *fresh, int n, mha_stream stream);

/*
 * kv_pages_compact -- the pages that some sequence holds, in increasing page
 * number, become pages 0 .. n_live-1 of other pools (of another size, or as
 * large), and the page tables are renumbered.  A shared page is moved once
 * and stays shared.  Ending a sequence is setting its length to 0: its pages
 * are then free unless another sequence holds them.
 *   src : the cache.  dst : the pools and page table to fill; its dtype,
 *       page_size, kv_heads, d, layers and B are src's, table_cols at least
 *       src's; num_pages and strides are its own, kv_lengths is not used.
 *       It must share no memory with src.
 *   n_live : device int32, the number of pages held.
 *   workspace : device, 16-byte aligned, at least
 *       kv_pages_compact_workspace_bytes(src->num_pages) bytes; one call's at
 *       a time, as above.
 * Entries of dst's table behind a sequence's last page, and pages from n_live
 * on, are left as they were.
 * Checked on the device (MHA_ERR_DEVICE): a length outside [0,
 * table_cols*page_size] (the sequence counts as empty), a page number outside
 * [0, num_pages) or a page without room in dst (its entry becomes -1).
 * src->num_pages <= 2^20.
 * Returns MHA_OK, MHA_ERR_INVALID_ARG, MHA_ERR_UNSUPPORTED or MHA_ERR_CUDA.
 */
mha_status kv_pages_compact(const mha_kv_pages *src, const mha_kv_pages *dst,
                            int32_t *n_live, void *workspace,
                            size_t workspace_bytes, mha_stream stream);

/* Workspace kv_pages_compact needs, in bytes (0 for a bad num_pages). */
size_t kv_pages_compact_workspace_bytes(int num_pages);

/* kv_pages_compact_e4m3 -- kv_pages_compact of a cache in 8 bits: the scales
 * move with their pages.  dst_scales shares no memory with src_scales. */
mha_status kv_pages_compact_e4m3(const mha_kv_pages *src,
                                 const mha_kv_scales *src_scales,
                                 const mha_kv_pages *dst,
                                 const mha_kv_scales *dst_scales,
                                 int32_t *n_live, void *workspace,
                                 size_t workspace_bytes, mha_stream stream);

/*
 * Attention over a long cache can leave most pages out.  Every full page has
 * bounds of its keys, column by column; a query's bounds of its scores with a
 * page's keys then cost two rows in place of page_size; each query takes the
 * pages with the largest ones.
 *   bounds      : device int8 [layers, num_pages, kv_heads, 2, d], dense,
 *                 16-byte aligned: lo, hi
 *   bound_scale : device fp32 [layers, num_pages, kv_heads], dense
 * with lo * bound_scale <= K <= hi * bound_scale over the page's rows.
 *
 * kv_pages_bounds -- the bounds of every page that the newest tokens
 * [q_offsets[b], q_offsets[b+1]) have filled or lie in and that is full:
 *   s = the smallest power of two >= 2^-100 with max |c| <= 127 s, 0 for zeros
 *   lo = floor(min c / s), hi = ceil(max c / s) by columns;  bound_scale = s
 * where c are the page's keys, or of a cache in 8 bits its codes, and
 * bound_scale is s times the page's key scale.  Called after each append (of
 * whole sequences at first: q_offsets from their lengths) it keeps the bounds
 * of all full pages; pages that are shared keep theirs, and a page that a fork
 * copies gets its own once it is full.  A compaction moves pages, not bounds:
 * after it they are made anew, for whole sequences.
 *   scales : of a cache in 8 bits (dtype MHA_E4M3); NULL for MHA_BF16.
 *   T : the packed tokens, q_offsets as for sdpa_paged.
 * d is 64 or 128.  Keys must be finite.
 * Checked on the device (MHA_ERR_DEVICE): kv_lengths[b] in [n_b,
 * table_cols*page_size], offsets ascending in [0, T], page numbers -- such a
 * sequence's or page's bounds are left as they were.
 * Returns MHA_OK, MHA_ERR_INVALID_ARG, MHA_ERR_UNSUPPORTED or MHA_ERR_CUDA.
 */
mha_status kv_pages_bounds(const mha_kv_pages *pages,
                           const mha_kv_scales *scales, int layer,
                           const int32_t *q_offsets, int T, int8_t *bounds,
                           float *bound_scale, mha_stream stream);

/*
 * kv_pages_select -- for every new token and kv head, n_select of the pages
 * that hold keys the token sees (causal, bottom-right, as in sdpa_paged): its
 * newest page, and of the full ones before it those with the largest score,
 * equal scores from the sequence's beginning on:
 *   qi = q / s to the nearest whole number, ties to even, s the smallest power
 *        of two >= 2^-100 with max |q| <= 127 s over the head's row
 *   score = max over the kv head's query heads of
 *           s * sum_c (max(qi_c, 0) hi_c + min(qi_c, 0) lo_c) * bound_scale
 * (a sum of max(qi_c lo_c, qi_c hi_c), as lo <= hi).
 * The sums are whole numbers, the products in fp32 in that order, so equal
 * calls select equal pages on every device.  Elements of q that are not
 * finite count as 0; a product beyond fp32 is an infinity, and one of those
 * with a bound_scale of 0 counts least.
 *   Q : bf16, T packed tokens as for sdpa_paged.
 *   bounds, bound_scale : of all the layers; `layer` picks.
 *   selected : device int32 [T, kv_heads, n_select], page numbers in the order
 *       of their positions, -1 behind the last.
 *   lengths : device int32 [T], the rows that the token sees in its selected
 *       pages (all full but the newest); 0 for a token of no sequence, -1
 *       where an entry is bad (selected then holds -1).
 *   workspace : device, 16-byte aligned, at least
 *       kv_pages_select_workspace_bytes(...) bytes; one call's at a time.
 * The pools are not read (their pointers are checked as anywhere): of *pages
 * num_pages, page_size, kv_heads, d, layers and the tables count.  d is 64 or 128, H / kv_heads <= 128, 1 <= n_select <=
 * 65536.
 * Checked on the device (MHA_ERR_DEVICE): kv_lengths[b] in [n_b,
 * table_cols*page_size], the page numbers a token sees, offsets ascending in
 * [0, T].
 * Returns MHA_OK, MHA_ERR_INVALID_ARG, MHA_ERR_UNSUPPORTED or MHA_ERR_CUDA.
 */
mha_status kv_pages_select(const void *Q, int64_t q_token_stride,
                           const mha_kv_pages *pages, int layer,
                           const int32_t *q_offsets, const int8_t *bounds,
                           const float *bound_scale, int T, int H,
                           int n_select, int32_t *selected, int32_t *lengths,
                           void *workspace, size_t workspace_bytes,
                           mha_stream stream);

/* Workspace kv_pages_select needs, in bytes (0 for bad sizes). */
size_t kv_pages_select_workspace_bytes(int T, int kv_heads, int table_cols);

/*
 * sdpa_paged_selected -- attention of T tokens, each over its own pages per kv
 * head: token t and kv head g see the first lengths[t] rows of the pages
 * selected[t, g, :], which kv_pages_select has filled (any table of that
 * layout will do).
 *   Q, O, H, scale, layer, out_dtype, num_splits : as for sdpa_paged.
 *   pages : the pools; its tables are not used (checked as anywhere: with B = 0
 *       and table_cols = 1 there need be none).
 *   scales : of a cache in 8 bits (dtype MHA_E4M3, whose operands are as in
 *       sdpa_paged_e4m3); NULL for MHA_BF16.
 *   selected : device int32 [T, kv_heads, n_select]; lengths : device int32
 *       [T].  A token of length 0 is passed over: its row of O stays as it was.
 * Checked on the device (MHA_ERR_DEVICE, the token's rows written as zeros):
 * lengths in [0, n_select*page_size], page numbers.
 * d is 64 or 128, H / kv_heads <= 128, n_select * page_size <= 2^30.
 * Returns MHA_OK, MHA_ERR_INVALID_ARG, MHA_ERR_UNSUPPORTED or MHA_ERR_CUDA.
 */
mha_status sdpa_paged_selected(const void *Q, int64_t q_token_stride,
                               const mha_kv_pages *pages,
                               const mha_kv_scales *scales, int layer,
                               const int32_t *selected, const int32_t *lengths,
                               int n_select, void *O, int T, int H,
                               float scale, mha_dtype out_dtype,
                               int num_splits, mha_stream stream);

/*
 * mha_create -- allocate a multi-head attention layer handle.
 *   d_model   : model width D.
 *   dtype     : element type of x, W and out (MHA_BF16 or MHA_F32).
 *   max_batch, max_lq, max_lk : the largest B, Lq, Lk later calls may use;
 *               they size the device workspace the handle owns
 *               (Q [B,H,Lq,d], K and V [B,H,Lk,d], context [B,Lq,D]).
 * The handle allocates that workspace with cudaMalloc on the current device
 * and frees it in mha_destroy.  *out is set to NULL on failure.
 * Returns MHA_OK, MHA_ERR_INVALID_ARG, MHA_ERR_OOM or MHA_ERR_CUDA.
 */
mha_status mha_create(mha_handle *out, int d_model, mha_dtype dtype,
                      int max_batch, int max_lq, int max_lk);

/*
 * mha_forward -- one multi-head attention layer forward.
 *   x_q  [B, Lq, D], x_kv [B, Lk, D] (x_kv may equal x_q: self-attention;
 *        a different tensor: cross-attention, keys/values from x_kv)
 *   Wq, Wk, Wv, Wo [D, D] row-major, applied as y = x @ W
 *   h    : number of heads; D % h must be 0; d = D / h.
 *   mask_kind, key_lengths : as for sdpa_forward.
 *   out  [B, Lq, D]
 * The projections write Q, K, V in [B, h, L, d] (the head split is the
 * store layout); attention writes the context in [B, Lq, D] (the concat is
 * the store layout); the output projection reads it.  Four launches on
 * `stream`.  Supported: BF16 with d in {64, 128}; F32 with d <= 128.
 * Returns MHA_OK, MHA_ERR_INVALID_ARG (incl. B/Lq/Lk above the handle's
 * maxima), MHA_ERR_UNSUPPORTED or MHA_ERR_CUDA.
 */
mha_status mha_forward(mha_handle handle, const void *x_q, const void *x_kv,
                       const void *Wq, const void *Wk, const void *Wv,
                       const void *Wo, int B, int Lq, int Lk, int h,
                       int mask_kind, const int32_t *key_lengths, void *out,
                       mha_stream stream);

/*
 * mha_forward_noalloc -- mha_forward for callers that cannot allocate device
 * memory.  (This entry point has no counterpart in the pages that define
 * the method; it is a property of this library's interface.)
 *
 * mha_forward keeps the projected Q, K, V and the concatenated-heads context
 * in workspace that mha_create allocates with cudaMalloc.  Callers that must
 * not call cudaMalloc -- a host program that gives all device memory to its
 * own pool, a plugin whose execution step may not allocate, a latency-bound
 * loop that cannot take cudaMalloc's implicit synchronisation -- call this
 * instead: the same four launches, with those intermediates in a fixed
 * device array inside the library.  It calls no cudaMalloc, cudaFree or
 * other allocating routine.
 *   d_model, dtype : as for mha_create; the other arguments as for
 *                    mha_forward.
 * Limit: the intermediates need 2*B*Lq*D + 2*B*Lk*D elements (each tensor
 * rounded up to 256 bytes); a call needing more than
 * MHA_NOALLOC_SCRATCH_BYTES returns MHA_ERR_INVALID_ARG and launches
 * nothing.
 * The array is held on every GPU that loads the library until the process
 * exits.  The first call on a device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current; make that first call
 * before any stream capture on the device.  All calls on a device share the
 * array and leave their intermediates in it; calls whose executions overlap
 * on the GPU (different streams without ordering) race on it.
 * Returns MHA_OK, MHA_ERR_INVALID_ARG, MHA_ERR_UNSUPPORTED or MHA_ERR_CUDA.
 */
#define MHA_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)
mha_status mha_forward_noalloc(int d_model, mha_dtype dtype, const void *x_q,
                               const void *x_kv, const void *Wq,
                               const void *Wk, const void *Wv, const void *Wo,
                               int B, int Lq, int Lk, int h, int mask_kind,
                               const int32_t *key_lengths, void *out,
                               mha_stream stream);

/*
 * One post-norm Transformer encoder layer (next to the attention layer it
 * contains):
 *   a   = MultiHead(x, x, x) with biases (as mha_forward, plus bq, bk, bv
 *         added to the projections and bo to the output projection)
 *   x1  = LayerNorm(x + a) * ln1_gamma + ln1_beta
 *   f   = max(0, x1 W1 + b1) W2 + b2
 *   out = LayerNorm(x1 + f) * ln2_gamma + ln2_beta
 * LayerNorm over each position's D values, population variance, ln_eps
 * added to the variance (PyTorch's default is 1e-5).
 *   -- "The Transformer" (hoshank.vercel.app), "The Mathematics" (FFN and
 *      output = LayerNorm(x + Sublayer(x))); "The Transformer" (rayaq.ca),
 *      "The feed-forward block", "Residuals and LayerNorm", "The encoder
 *      stack" and the EncoderLayer of "Implementation".
 * All parameters have the layer's element type and are device pointers,
 * 16-byte aligned; matrices are row-major [d_in, d_out] applied as y = x@W.
 */
typedef struct {
    const void *Wq, *Wk, *Wv, *Wo;     /* [D, D] */
    const void *bq, *bk, *bv, *bo;     /* [D] */
    const void *ln1_gamma, *ln1_beta;  /* [D] */
    const void *W1;                    /* [D, F] */
    const void *b1;                    /* [F] */
    const void *W2;                    /* [F, D] */
    const void *b2;                    /* [D] */
    const void *ln2_gamma, *ln2_beta;  /* [D] */
} mha_encoder_params;

typedef struct mha_encoder_ctx *mha_encoder;

/* encoder_create -- a layer handle for d_model D, `heads`, FFN width d_ff,
 * element type `dtype`, up to max_batch x max_len tokens; owns cudaMalloc'd
 * workspace (Q, K, V, context, two [B,L,D] temporaries, x1, the [B,L,F]
 * hidden activation).  Supported: BF16 with D/heads in {64, 128} and D, d_ff
 * multiples of 64; F32 with D/heads <= 128; D <= 4096.  Returns MHA_OK,
 * MHA_ERR_INVALID_ARG, MHA_ERR_UNSUPPORTED, MHA_ERR_OOM or MHA_ERR_CUDA. */
mha_status encoder_create(mha_encoder *out, int d_model, int heads, int d_ff,
                          mha_dtype dtype, int max_batch, int max_len);

/* encoder_forward -- out [B, L, D] = layer(x [B, L, D]); mask_kind and
 * key_lengths as for mha_forward (self-attention, Lq = Lk = L).
 * out_dtype is the element type of `out`: the layer's type, or MHA_F32 for
 * a BF16 layer (the final LayerNorm's output stored unrounded).  BF16
 * layers with D <= 512 take five launches on `stream` (the residual add and
 * LayerNorm run in the epilogues of the W^O and W2 GEMMs, so the sublayer
 * outputs stay fp32 and are never stored); other layers take seven.  The
 * hidden activation and x1 are stored in the layer's type.  out must not
 * alias x.  Returns MHA_OK, MHA_ERR_INVALID_ARG or MHA_ERR_CUDA. */
mha_status encoder_forward(mha_encoder enc, const void *x,
                           const mha_encoder_params *params, int B, int L,
                           int mask_kind, const int32_t *key_lengths,
                           float ln_eps, void *out, mha_dtype out_dtype,
                           mha_stream stream);

/* encoder_destroy -- free the handle (synchronises the device).  NULL is
 * accepted. */
mha_status encoder_destroy(mha_encoder enc);

/*
 * mha_check -- synchronise the current device and report (then clear) its
 * device-side error word.  `handle` may be NULL.  Returns MHA_OK,
 * MHA_ERR_TIMEOUT, MHA_ERR_DEVICE or MHA_ERR_CUDA.
 */
mha_status mha_check(mha_handle handle);

/*
 * mha_selftest_wait_timeout -- exercise the failure path of the kernels'
 * bounded waits: launches one warp that waits on a shared-memory mbarrier
 * nothing arrives on, using the same wait routine as the attention and GEMM
 * pipelines, with a limit of `limit_ms` (1..10000).  The wait gives up, the
 * kernel sets MHA_ERR_TIMEOUT in the device error word and returns; a later
 * mha_check() reports (and clears) it and the context stays usable.  (A
 * property of this library's interface; the pages have no counterpart.)
 * Returns MHA_OK (launched), MHA_ERR_INVALID_ARG or MHA_ERR_CUDA.
 */
mha_status mha_selftest_wait_timeout(int limit_ms, mha_stream stream);

/* mha_destroy -- free the handle and its workspace (synchronises the
 * device first).  NULL is accepted. */
mha_status mha_destroy(mha_handle handle);

/* Static, NUL-terminated name of a status code. */
const char *mha_status_string(mha_status status);

/* Set the time limit, in milliseconds, after which a kernel pipeline wait
 * gives up and reports MHA_ERR_TIMEOUT (default 2000; applies to later
 * launches).  Returns the previous value. */
int mha_set_wait_limit_ms(int ms);

#ifdef __cplusplus
}
#endif

#endif /* GB300_MHA_H */
