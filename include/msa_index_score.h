/*
 * msa_index_score.h -- C ABI of the MSA index-branch block-score operator for
 * AMD Instinct MI355X (gfx950).
 *
 * The operator (gitcode cann/ops-transformer issue #4117 "MsaIndexScore",
 * section 计算过程; xxmr.cn guide to cann_ops_transformer.msa_index_score,
 * sections 二, 四, 五) computes, for every packed query token t of request b,
 * every index head h and every logical KV block beta of P = 128 tokens:
 *
 *   score[h, t, beta] = max_{j in block beta, j <= q_pos(t), j < kv_len[b]}
 *                       < query[t, h, :], k~[j, h / g, :] >
 *
 * with g = Hq / Hkv, q_pos(t) = kv_len[b] - L_q(b) + (t - cu_seqlens_q[b])
 * under the right-down causal mode (sparse_mode 3) and kv_len[b] - 1 without a
 * causal mask (sparse_mode 0).  k~ is the key row of logical block beta: for a
 * paged key it lives in physical page block_table[b, beta]; for a packed (TND)
 * key it is token sum_{b' < b} kv_len[b'] + j.  For an int8 key the dot product
 * is multiplied by scale[page, h_kv, j mod P] (TND: scale[token, h_kv]) before
 * the mask and the maximum (issue #4117: DOT -> DEQUANT -> MASK -> MAX).
 * Blocks with no visible key score -inf, requests with kv_len = 0 score -inf
 * everywhere, and output columns past a request's block count up to the
 * output width are -inf.  Then local_mask (guide, section 二) writes 1e30f on
 * blocks [0, init_blocks) and 1e29f on [max(0, start_loc[b]+1-local_blocks),
 * start_loc[b]] (the latter overriding), unless both counts are 0.  The output
 * is float32 [Hq, T, RoundUp(MB, 16)] (guide, section 五).
 *
 * No torch or HIP types appear here: pointers are plain device pointers and
 * the stream is a hipStream_t passed as void* (NULL = the null stream).
 */
#ifndef MSA_INDEX_SCORE_H
#define MSA_INDEX_SCORE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes.  Every check runs on the host before any device work; on a
 * non-zero status nothing is launched and `out` is untouched. */
typedef enum {
  MSA_OK = 0,
  MSA_ERR_NULL = 1,    /* a required pointer is NULL */
  MSA_ERR_LAYOUT = 2,  /* layout is not TND, BBND or BNBD (guide, section 三) */
  MSA_ERR_DTYPE = 3,   /* unsupported query/key element types (guide, section 七) */
  MSA_ERR_SHAPE = 4,   /* shapes disagree with each other or with the layout */
  MSA_ERR_STRIDE = 5,  /* a key axis other than dim0 is not compact (guide, 8.1) */
  MSA_ERR_SCALE = 6,   /* int8 key without scale, or scale with a non-int8 key */
  MSA_ERR_ATTR = 7,    /* sparse_mode not 0/3, init/local_blocks out of range, or
                          another attribute (family, local_mode, top-k k) invalid */
  MSA_ERR_HIP = 8,     /* a HIP runtime call or kernel launch failed */
  MSA_ERR_WORKSPACE = 9 /* the workspace is smaller than the call needs */
} msa_status_t;

/* Key layouts (guide, section 四): packed [T2, Hkv, D]; paged
 * [NP, P, Hkv, D] (BBND) and [NP, Hkv, P, D] (BNBD). */
typedef enum { MSA_LAYOUT_TND = 0, MSA_LAYOUT_BBND = 1, MSA_LAYOUT_BNBD = 2 } msa_layout_t;

/* For msa_cache_append only: a destination [T, H, D] with one row per new
 * token and head (rotated or encoded queries), not a cache. */
#define MSA_LAYOUT_ROWS 3

/* Where local_mask's window of local_blocks blocks ends.  PER_REQUEST: at
 * start_loc[b] for every token of request b (guide, section 二).  PER_QUERY:
 * at each query token's own block, floor(pos / 128) with pos = kv_len[b] -
 * L_q(b) + i the token's position in the sequence -- the paper's forced local
 * block b_local(i) (notes "MiniMax Sparse Attention: paper algorithm and
 * code", section 4.7, which observes that a request-wide window is not the
 * same in a long prefill).  A token before position 0 gets no window. */
typedef enum { MSA_LOCAL_PER_REQUEST = 0, MSA_LOCAL_PER_QUERY = 1 } msa_local_mode_t;

/* Element types.  Supported (query, key) pairs: (F16, F16), (BF16, BF16),
 * (F16, I8) with a float32 scale, (F8E4M3, F8E4M3) and (F8E5M2, F8E5M2)
 * (guide, section 七: int8 needs an fp16 query; FP8 query and key of one type,
 * no scale).  F8E4M3 is OCP e4m3 "fn" (finite, max 448); F8E5M2 is OCP e5m2. */
typedef enum {
  MSA_DTYPE_F16 = 0,
  MSA_DTYPE_BF16 = 1,
  MSA_DTYPE_I8 = 2,
  MSA_DTYPE_F8E4M3 = 3,
  MSA_DTYPE_F8E5M2 = 4,
  MSA_DTYPE_MXFP4 = 5  /* E2M1 pairs, one byte each; see msa_index_score_mxfp4 */
} msa_dtype_t;

/* A strided view of device memory.  `data` points at element [0, 0, ...];
 * `stride` is in elements.  Only the first `ndim` entries are read. */
typedef struct {
  const void* data;
  int32_t dtype;       /* msa_dtype_t */
  int32_t ndim;
  int64_t shape[4];
  int64_t stride[4];
} msa_tensor_t;

/*
 * Compute the block scores.
 *
 * query        [T, Hq, D] compact; D must be 128.
 * key          TND [T2, Hkv, D] fully compact; BBND [NP, P, Hkv, D] or
 *              BNBD [NP, Hkv, P, D] with P = 128, any dim0 stride (pages may
 *              sit apart in memory, guide 8.1), other axes of extent > 1
 *              compact (extent-1 axes are not addressed, so their stride is
 *              ignored).  A 3-D BBND key [NP, P, D] means Hkv = 1.
 * start_loc    device int32 [B]: logical block index of the request's current
 *              query (guide, section 四); used only by local_mask.
 * block_table  device int32 [B, max_blocks] row-major, paged layouts only
 *              (NULL for TND).  Entries at or past a request's block count
 *              ceil(kv_len/128) are never read.
 * max_blocks   MB: the block_table width for paged layouts; for TND the
 *              largest ceil(kv_len[b]/128) over the batch (an all-empty batch
 *              may pass 0 or 1).
 * scale        device float32, int8 keys only (NULL otherwise): paged
 *              [NP, Hkv, P] indexed by logical page number, TND [T2, Hkv].
 * cu_seqlens_q device int32 [B+1], cu_seqlens_q[0] = 0, non-decreasing,
 *              cu_seqlens_q[B] = T.
 * kv_len       device int32 [B], visible KV length of each request (for TND
 *              the requests' keys are packed back to back in this order;
 *              the guide's TND actual_seq_klen is the [B+1] prefix sum of
 *              these lengths, which the caller differences first).
 * batch        B, the number of requests (>= 0; 0 only when T = 0).
 * block_size   tokens per logical block, which is also a paged key's P axis
 *              (guide, section 四: the kernel splits every request's keys into
 *              blocks of block_size = 128); must be 128 (MSA_ERR_SHAPE
 *              otherwise).
 * layout       msa_layout_t.
 * sparse_mode  3 (right-down causal) or 0 (no causal mask).
 * init_blocks, local_blocks
 *              local_mask counts, each in [0, limit] with limit = MB for
 *              paged layouts and RoundUp(MB,16) for TND (guide, section 十).
 * out          device float32 [Hq, T, out_width], compact, written in full.
 * out_width    must equal msa_index_score_out_width(max_blocks).
 * stream       hipStream_t (as void*); the call is asynchronous on it.
 *
 * Device-data preconditions (the caller's contract, not checked on device):
 * the cu_seqlens_q rules above; paged: kv_len[b] <= MB*128 and
 * block_table[b, beta] in [0, NP) for beta < ceil(kv_len[b]/128); TND:
 * sum(kv_len) = T2 and ceil(kv_len[b]/128) <= MB.  Blocks at or past MB are
 * never scored or read, whatever kv_len says.
 *
 * NULL is accepted for pointers the call cannot read: kv_len, start_loc and
 * block_table when batch = 0, and out when T = 0.
 *
 * Ownership: every pointer is caller-owned; the library allocates no device
 * memory.  The only state it keeps between calls is one figure per device,
 * key type and batch kind (at most 64 requests, or more): the decode
 * kernel's workgroup slot count (CU count times occupancy), asked of the HIP
 * runtime on the first such decode launch on that device (read and written
 * atomically).  Calls may overlap, from several host threads and on the same
 * or different streams: they share no device memory.  Returns MSA_OK
 * or an error status; T = 0 returns MSA_OK without launching anything.
 * MSA_ERR_HIP reports a failure of this call's own runtime queries or
 * launch, never an error pending from earlier HIP work.  query, key and out
 * must be 16-byte aligned and a paged key's dim0 stride a multiple of 16
 * bytes (MSA_ERR_STRIDE otherwise).  Sizes past the kernels' 32-bit indexing
 * return MSA_ERR_SHAPE: out_width > 2^24, Hq > 2^16, batch > 2^30, T >= 2^31,
 * or one 128-token block of one head spanning 2 GiB or more of key memory.
 */
msa_status_t msa_index_score(const msa_tensor_t* query, const msa_tensor_t* key,
                             const int32_t* start_loc, const int32_t* block_table,
                             int64_t max_blocks, const float* scale,
                             const int32_t* cu_seqlens_q, const int32_t* kv_len,
                             int32_t batch, int32_t block_size, int32_t layout,
                             int32_t sparse_mode, int32_t init_blocks, int32_t local_blocks,
                             float* out, int64_t out_width, void* stream);

/* Same as msa_index_score, with the kernel family chosen by the caller:
 * family = -1 picks it from the sizes (as msa_index_score does), 0 forces the
 * decode tiles, 1 the prefill tiles.  Both families compute the same
 * definition for every valid input; the choice only changes speed.  Any other
 * family value returns MSA_ERR_ATTR.  For tests and benchmarks. */
msa_status_t msa_index_score_family(const msa_tensor_t* query, const msa_tensor_t* key,
                                    const int32_t* start_loc, const int32_t* block_table,
                                    int64_t max_blocks, const float* scale,
                                    const int32_t* cu_seqlens_q, const int32_t* kv_len,
                                    int32_t batch, int32_t block_size, int32_t layout,
                                    int32_t sparse_mode, int32_t init_blocks,
                                    int32_t local_blocks, float* out, int64_t out_width,
                                    void* stream, int32_t family);

/* Same as msa_index_score_family, with the local_mask window's placement
 * chosen by local_mode (msa_local_mode_t; any other value returns
 * MSA_ERR_ATTR).  With MSA_LOCAL_PER_QUERY start_loc is not read and may be
 * NULL; everything else (arguments, ownership, errors) is as for
 * msa_index_score.  msa_index_score is this call with MSA_LOCAL_PER_REQUEST
 * and family -1. */
msa_status_t msa_index_score_ex(const msa_tensor_t* query, const msa_tensor_t* key,
                                const int32_t* start_loc, const int32_t* block_table,
                                int64_t max_blocks, const float* scale,
                                const int32_t* cu_seqlens_q, const int32_t* kv_len,
                                int32_t batch, int32_t block_size, int32_t layout,
                                int32_t sparse_mode, int32_t init_blocks, int32_t local_blocks,
                                int32_t local_mode, float* out, int64_t out_width, void* stream,
                                int32_t family);

/* The block score on MXFP4 index vectors: the FP4 indexer variant of the
 * notes "MiniMax Sparse Attention: paper algorithm and code" (section 4.6,
 * path B, and section 8.2: MXFP4 is E2M1 values with an E8M0 scale per group
 * of elements, the block scores stay float32).  Same definition as
 * msa_index_score, with q and k~ the decoded MXFP4 vectors: element d of a
 * row is its E2M1 value times 2^(s - 127), s the E8M0 scale byte of group
 * d / 32 (E2M1: sign, 2 exponent bits with bias 1, 1 fraction bit; exponent
 * 0 gives 0 or 0.5; largest 6.  E8M0 255 is NaN).  The product is exact in
 * the MFMA's float32 accumulation up to summation rounding; the result
 * approximates the higher-precision score only as far as the encoding does.
 *
 * query        dtype MSA_DTYPE_MXFP4, [T, Hq, 64] bytes (128 elements, two per
 *              byte, the even element in the low nibble), compact, 16-byte
 *              aligned.
 * query_scale  device uint8 [T, Hq, 4] compact: E8M0 of elements 32c..32c+31.
 * key          dtype MSA_DTYPE_MXFP4, layouts as msa_index_score with a last
 *              axis of 64 bytes: TND [T2, Hkv, 64], BBND [NP, 128, Hkv, 64],
 *              BNBD [NP, Hkv, 128, 64]; paged dim0 stride any multiple of 16
 *              bytes.
 * key_scale    device uint8, compact, the key's layout with a last axis of 4:
 *              TND [T2, Hkv, 4], BBND [NP, 128, Hkv, 4], BNBD [NP, Hkv, 128, 4],
 *              indexed by page number (whatever the key's dim0 stride);
 *              4-byte aligned, like query_scale.
 * local_mode   msa_local_mode_t.  Everything else as msa_index_score.
 *
 * The kernel family is picked from the sizes, as msa_index_score does.
 * Returns as msa_index_score, plus MSA_ERR_DTYPE unless query and key are
 * MSA_DTYPE_MXFP4 and MSA_ERR_NULL for a NULL scale when T > 0 (with no
 * query tokens nothing is read and both scales may be NULL).  (msa_index_score and
 * its variants return MSA_ERR_SCALE for MXFP4 tensors: they cannot carry the
 * group scales.) */
msa_status_t msa_index_score_mxfp4(const msa_tensor_t* query, const uint8_t* query_scale,
                                   const msa_tensor_t* key, const uint8_t* key_scale,
                                   const int32_t* start_loc, const int32_t* block_table,
                                   int64_t max_blocks, const int32_t* cu_seqlens_q,
                                   const int32_t* kv_len, int32_t batch, int32_t block_size,
                                   int32_t layout, int32_t sparse_mode, int32_t init_blocks,
                                   int32_t local_blocks, int32_t local_mode, float* out,
                                   int64_t out_width, void* stream);

/* Same as msa_index_score_mxfp4, with the kernel family chosen by the caller
 * as for msa_index_score_family (-1 from the sizes, 0 the decode tiles, 1 the
 * prefill tiles; any other value returns MSA_ERR_ATTR).  For tests and
 * benchmarks. */
msa_status_t msa_index_score_mxfp4_family(const msa_tensor_t* query, const uint8_t* query_scale,
                                          const msa_tensor_t* key, const uint8_t* key_scale,
                                          const int32_t* start_loc, const int32_t* block_table,
                                          int64_t max_blocks, const int32_t* cu_seqlens_q,
                                          const int32_t* kv_len, int32_t batch,
                                          int32_t block_size, int32_t layout,
                                          int32_t sparse_mode, int32_t init_blocks,
                                          int32_t local_blocks, int32_t local_mode, float* out,
                                          int64_t out_width, void* stream, int32_t family);

/* Top-k block selection on the score rows: the stage the pages place after
 * the block score (the notes "MiniMax Sparse Attention: paper algorithm and
 * code", section 4.7 "Top-k Block
 * Selection", section 5.3 "Top-k" with the sparse_topk_select contract,
 * section 6.1 "Exp-free Top-k").
 *
 * For every query token t and index head h, among the blocks beta < num_valid
 * of the row scores[h, t, :] whose score is above -inf (NaN never qualifies),
 * the k with the highest scores, equal scores taken by lower block index,
 * are written to out[t, h, 0:k] in ascending block order; the slots past the
 * number selected hold -1.  Selection works on the raw scores, compared as
 * floats (so -0.0 and +0.0 are equal scores).
 *
 * scores     device float32 [Hq, T, width], compact (msa_index_score's out),
 *            4-byte aligned; not read when num_valid = 0.
 * Hq, T, width  sizes, >= 0, Hq <= 65535, T <= 2^33, width <= 2^24, and
 *            Hq * T * width below 2^63.
 * num_valid  blocks to consider, in [0, width] (the table width MB for an
 *            msa_index_score output; columns past it are padding).
 * k          1..64 (the sparse_topk_select contract uses 16).
 * out        device int32 [T, Hq, k], compact, 4-byte aligned, written in full.
 * stream     hipStream_t (as void*); the call is asynchronous on it.
 *
 * Ownership: caller-owned pointers; nothing is allocated or kept.  Returns
 * MSA_OK (also, without launching or checking pointers, when Hq * T = 0),
 * MSA_ERR_SHAPE for sizes out of range, MSA_ERR_ATTR for k out of range,
 * MSA_ERR_NULL for a NULL pointer the call must use, MSA_ERR_STRIDE for a
 * misaligned one, MSA_ERR_HIP if the launch fails. */
msa_status_t msa_block_topk(const float* scores, int64_t Hq, int64_t T, int64_t width,
                            int64_t num_valid, int32_t k, int32_t* out, void* stream);

/* ---------------------------------------------------------------------------
 * Around the index branch: the cache append that comes before the block score
 * and the attention that comes after the selection.
 *
 * Shared by the entry points below.  Token t of request b (cu_seqlens_q[b] <=
 * t < cu_seqlens_q[b+1]), the i-th of its L_q(b) new tokens, stands at
 * position pos(t) = kv_len[b] - L_q(b) + i: kv_len counts the new tokens.
 * cu_seqlens_q, kv_len, block_table, max_blocks, batch, block_size (128) and
 * stream are as for msa_index_score, except that
 *  - cu_seqlens_q[B] may be less than T: rows of tokens behind the last
 *    request (a padded batch) are neither read nor written;
 *  - a table entry outside [0, NP) names no page: nothing is written there,
 *    and its keys are not visible;
 *  - max_blocks <= 2^24, batch <= 2^30, T < 2^31, at most 2^16 heads, at most
 *    2^31 - 1 pages or packed keys, one 128-token block of one head spans less
 *    than 2 GiB, and a launch holds less than 2^32 threads (reached from about
 *    2 million tokens at 8 KV heads on; MSA_ERR_SHAPE otherwise).
 * Blocks at or past max_blocks, and packed keys past the tensor's end, are
 * neither read nor written, whatever kv_len says.  All pointers are
 * caller-owned, nothing is allocated or kept, calls may overlap as long as
 * they write different memory, and they may be captured into HIP graphs (two
 * graphs that may run at once need workspaces of their own).  T = 0 returns
 * MSA_OK without launching anything.
 * ------------------------------------------------------------------------ */

/* One tensor of a msa_cache_append call. */
typedef struct {
  msa_tensor_t src;   /* [T, H, 128] f16 or bf16: any token and head strides of
                         whole 16 bytes, the last axis compact */
  msa_tensor_t dst;   /* where the rows go, see below */
  void* scale;        /* the scales that an int8 or MXFP4 dst needs, else NULL */
  int32_t layout;     /* msa_layout_t of a cache, or MSA_LAYOUT_ROWS */
  int32_t rotate;     /* 1: the rows are rotated first; 0: stored as they are */
} msa_append_item_t;

#define MSA_APPEND_MAX_ITEMS 8

/*
 * Append new tokens' rows to caches, rotated by their positions and encoded as
 * the cache holds them; and rotate or encode the queries in the same launch.
 *
 * For every item, token t and head h, y = src[t, h, :], rotated if asked for:
 * with c = cos[pos, r], s = sin[pos, r] and the r-th pair (a, b) of the first
 * rotary_dim elements -- elements (r, r + rotary_dim / 2), or (2r, 2r + 1)
 * with interleaved = 1 --
 *     a' = a c - b s,   b' = b c + a s;
 * elements past rotary_dim stay as they are.  Then y is stored
 *  - in a paged cache (BBND [NP, 128, H, D], BNBD [NP, H, 128, D], strides as
 *    msa_index_score's key) in page block_table[b, pos / 128], slot pos % 128;
 *  - in a packed cache (TND [T2, H, D]) at token sum_{b' < b} kv_len[b'] + pos;
 *  - with MSA_LAYOUT_ROWS in dst[t, h, :] (strides as src, rows that do not
 *    overlap; may be src itself, if no other item reads that src).
 * dst's type says how:
 *  - src's own type: rounded to nearest even;
 *  - F8E4M3, F8E5M2: rounded to nearest even, past the largest finite value to
 *    that value, NaN kept;
 *  - I8: scale = max |y| / 127 (float32), element = y / scale rounded to
 *    nearest even.  scale: float32 [NP, H, 128] for both paged layouts,
 *    [T2, H] packed, [T, H] rows;
 *  - MXFP4 (last axis 64 bytes): per group of 32 elements E8M0 =
 *    floor(log2 max |y|) - 2 + 127 (at least 0), elements y / 2^(E8M0 - 127)
 *    rounded to the nearest E2M1 value, ties to the even code, past 6 to 6.
 *    scale: uint8, dst's layout with a last axis of 4, compact, 4-byte aligned.
 * The rotation for the last three is evaluated in float64, so that a value
 * next to a rounding border falls on its own side; a zero row or group has
 * scale 0 and zero elements; a row (I8) or group (MXFP4) that holds an
 * infinity or NaN gets a NaN scale (E8M0 255) and zero elements.  The encoded
 * types are the index branch's (msa_index_score and its variants read them);
 * msa_attention takes keys and values of the query's type.
 *
 * cos, sin     device float32 [positions, rotary_dim / 2], compact, 16-byte
 *              aligned; may be NULL if no item is rotated.
 * rotary_dim   a multiple of 16 in [16, 128] if any item is rotated.
 * interleaved  0 or 1, how elements pair up.
 * block_table  may be NULL if no item is a paged cache.
 *
 * A token before position 0, or (if any item is rotated) at or past
 * `positions`, is skipped in every item.  A call must not write one place
 * twice (two items with one dst, two requests' tables naming one page for new
 * tokens): which row stays is not defined.
 * Returns MSA_ERR_ATTR for num_items outside [1, MSA_APPEND_MAX_ITEMS] or a
 * bad rotate, rotary_dim or interleaved, MSA_ERR_SCALE for a scale given with
 * a type that has none or missing, MSA_ERR_DTYPE, _LAYOUT, _SHAPE, _STRIDE,
 * _NULL as msa_index_score does. */
msa_status_t msa_cache_append(const msa_append_item_t* items, int32_t num_items,
                              const float* cos, const float* sin, int64_t positions,
                              int32_t rotary_dim, int32_t interleaved,
                              const int32_t* block_table, int64_t max_blocks,
                              const int32_t* cu_seqlens_q, const int32_t* kv_len, int32_t batch,
                              int32_t block_size, void* stream);

#define MSA_APPEND_MAX_AXES 4

/*
 * The same with several position axes (time, height and width of an image's or
 * a video's tokens): pair r of token t is rotated by the angles of row
 * axis_positions[pair_axes[r], t] instead of the token's position in its
 * sequence, which still says where the row is stored.
 *
 * axis_positions  device int32 [axes, T], compact.
 * axes            1..MSA_APPEND_MAX_AXES (MSA_ERR_ATTR otherwise).
 * pair_axes       host uint8 [rotary_dim / 2]: the axis of each pair, below axes
 *                 (MSA_ERR_ATTR); read before the call returns.  Axes in runs of
 *                 pairs (0 0 .. 1 1 .. 2 2) or in turn (0 1 2 0 1 2 ..) are both
 *                 said this way.
 *
 * A token with any axis position outside [0, positions), or before position 0 of
 * its sequence, is skipped in every item; its position may be at or past
 * `positions`.  If no item is rotated, the axes are not looked at.  Everything else
 * as msa_cache_append.
 */
msa_status_t msa_cache_append_axes(const msa_append_item_t* items, int32_t num_items,
                                   const float* cos, const float* sin, int64_t positions,
                                   int32_t rotary_dim, int32_t interleaved,
                                   const int32_t* axis_positions, int32_t axes,
                                   const uint8_t* pair_axes, const int32_t* block_table,
                                   int64_t max_blocks, const int32_t* cu_seqlens_q,
                                   const int32_t* kv_len, int32_t batch, int32_t block_size,
                                   void* stream);

/*
 * Attention of the new tokens: over a paged cache (a chunk of a prompt, one
 * decode token, speculative tokens, or requests of each kind in one batch), or
 * over packed keys (whole prompts of different lengths).
 *
 *   S[t,h,j] = softmax_scale <query[t,h,:], key[j, h/g, :]>
 *   out[t,h,:] = sum_j exp(S - m) value[j, h/g, :] / sum_j exp(S - m)
 *   lse[t,h] = log sum_j exp(S)
 *
 * over the visible j: j < kv_len[b] and, with sparse_mode 3, j <= pos(t).  A
 * row that sees no key gets out 0 and lse -inf.  S, the softmax's maximum and
 * sum and both products' sums are float32; the weights exp(S - m) are rounded
 * to the query's type for the second product, and out once at the end.  (f16
 * weights are scaled first, so that the row's largest is at least 2^11: a key's
 * share is lost only below 2^-36 of it, 25 nats.)
 * Infinities and NaN in keys or values that a row does not see never reach it.
 * (The sums are taken before the division, with bf16 weights of up to 2^8 each:
 * n visible bf16 values past 2^120 / n in magnitude may give infinities.)
 *
 * query        f16 or bf16 [T, Hq, 128], any token stride >= Hq * 128 of whole
 *              16 bytes, other axes compact.
 * key, value   the query's type, layouts as msa_index_score's key, each with a
 *              page stride of its own; packed ones with any token stride >=
 *              Hkv * 128 of whole 16 bytes.  Hq a multiple of Hkv.
 * max_blocks   as for msa_index_score (packed: a bound on ceil(kv_len / 128);
 *              it only steers how the work is split).
 * softmax_scale  positive and finite (1 / sqrt(128) in most models).
 * out          device [T, Hq, 128] of the query's type, compact, 16-byte
 *              aligned.
 * lse          device float32 [T, Hq], compact, or NULL.
 * workspace    device memory of at least msa_attention_workspace(...) bytes,
 *              16-byte aligned, for this call alone until it has run; may be
 *              NULL if that is 0 (MSA_ERR_WORKSPACE if it is too small).
 * The same call gives the same bits every time. */
msa_status_t msa_attention(const msa_tensor_t* query, const msa_tensor_t* key,
                           const msa_tensor_t* value, const int32_t* block_table,
                           int64_t max_blocks, const int32_t* cu_seqlens_q, const int32_t* kv_len,
                           int32_t batch, int32_t block_size, int32_t layout, int32_t sparse_mode,
                           float softmax_scale, void* out, float* lse, void* workspace,
                           int64_t workspace_bytes, void* stream);

/*
 * The same with other scores, and other keys that a token sees.  In this order:
 *
 *   S1 = softcap tanh(S / softcap)       with softcap > 0
 *   S2 = S1 - slopes[h] |pos(t) - j|     with slopes
 *
 * take the place of S, and with `visible` token t sees only j with
 * visible[t, 0] <= j < visible[t, 1] among those that sparse_mode lets it see:
 * with mode 3 the documents of a packed sequence (a document's first key, and any
 * end past the token), with mode 0 images or prefixes whose tokens see each other
 * both ways (0, and the larger of pos(t) + 1 and the end of the token's image or
 * of the prefix).  Blocks that no token of a tile sees are not read.
 *
 * softcap      0 (none) or positive, finite; MSA_ERR_ATTR otherwise, and where
 *              softmax_scale / softcap has no float32.  Beside S's own error a capped
 *              score is off by 4 units in its last place at most where all scores of
 *              its tile are below 5/8 softcap, and by 6 units in the last place of the
 *              cap elsewhere (units of 2^-23).
 * slopes       device float32 [Hq], compact, finite; or NULL.  (Bias and scores are
 *              added in float32, with the biases taken against that of the nearest key
 *              that the token's range and sparse_mode leave: keys far behind that one
 *              lose digits that their weights do not have.)
 * visible      device int32 [T, 2], compact, 8-byte aligned; or NULL.  Any values: a
 *              token with visible[t, 1] <= visible[t, 0] sees nothing.  Rows of
 *              tokens behind the last request are not read.
 *
 * workspace    at least msa_attention's; with msa_attention_ex_workspace(...) bytes
 *              short calls are split into shorter parts (50 tokens over 2992 keys,
 *              capped: 44 us without, 30 with it).
 *
 * With none of the three it is msa_attention, bit for bit.  lse is the log of the
 * sum of exp(S2).  In tiles of the same rows whose keys are not split, a row's bits do
 * not depend on the rows computed beside it, nor on keys that it does not see, but for
 * capped scores, by the errors above.  Tiles and splits go by the sizes, the lengths,
 * the ranges and the workspace.
 */
msa_status_t msa_attention_ex(const msa_tensor_t* query, const msa_tensor_t* key,
                              const msa_tensor_t* value, const int32_t* block_table,
                              int64_t max_blocks, const int32_t* cu_seqlens_q,
                              const int32_t* kv_len, int32_t batch, int32_t block_size,
                              int32_t layout, int32_t sparse_mode, float softmax_scale,
                              float softcap, const float* slopes, const int32_t* visible,
                              void* out, float* lse, void* workspace, int64_t workspace_bytes,
                              void* stream);

/* msa_attention over selected blocks: j is visible to the heads of KV head h only
 * if also floor(j / 128) is among blocks[t, h, 0:num_blocks] (device int32
 * [T, Hkv, num_blocks], compact, num_blocks 1..64: msa_block_topk's output for
 * one index head per KV head).  Entries may stand in any order; one outside the
 * request's visible blocks (-1 among them) names nothing, and a block named
 * twice counts once. */
msa_status_t msa_block_attention(const msa_tensor_t* query, const msa_tensor_t* key,
                                 const msa_tensor_t* value, const int32_t* blocks,
                                 int32_t num_blocks, const int32_t* block_table,
                                 int64_t max_blocks, const int32_t* cu_seqlens_q,
                                 const int32_t* kv_len, int32_t batch, int32_t block_size,
                                 int32_t layout, int32_t sparse_mode, float softmax_scale,
                                 void* out, float* lse, void* workspace, int64_t workspace_bytes,
                                 void* stream);

/* Bytes of workspace that msa_attention (num_blocks = 0) or
 * msa_block_attention needs for a call of these sizes; 0 if it needs none.
 * Host-only. */
int64_t msa_attention_workspace(int64_t T, int32_t batch, int32_t Hq, int32_t Hkv,
                                int64_t max_blocks, int32_t num_blocks);

/* Bytes of workspace with which msa_attention_ex splits a call of these sizes as
 * it would choose to, whatever its form: msa_attention_workspace(..., 0) or more.
 * Host-only. */
int64_t msa_attention_ex_workspace(int64_t T, int32_t batch, int32_t Hq, int32_t Hkv,
                                   int64_t max_blocks);

/* Rows -- (query token, head) pairs of one KV head -- of the tiles that
 * msa_attention (num_blocks = 0) or msa_block_attention would use for a call of
 * these sizes: 16, 128 or 256; 0 for sizes that no call takes.  (msa_attention_ex
 * may take 128 where this says 256.)  All tiles compute the same definition.
 * Host-only; for benchmarks and tests. */
int32_t msa_attention_tile_rows(int64_t T, int32_t batch, int32_t Hq, int32_t Hkv,
                                int64_t max_blocks, int32_t num_blocks);

/*
 * The tables of one serving step, from the requests' lengths: what the entry
 * points here take as cu_seqlens_q, kv_len, start_loc and block_table, with
 * pages from a free list for the blocks that the new tokens begin, and every new
 * token's position and slot.  For request b with q = new_tokens[b], c =
 * ctx_len[b] (negative counts as 0), row r = rows[b] of the pool:
 *
 *   cu_seqlens_q[b + 1] = sum of the new tokens of requests 0..b
 *   kv_len[b] = c + q,  start_loc[b] = floor(c / 128)
 *   blocks ceil(c / 128) .. ceil(kv_len[b] / 128) - 1 take the next pages, in the
 *     order of b and then of the block, from the end of the free list:
 *     free_pages[n - 1], free_pages[n - 2], ... with n = free_count[0]; behind
 *     the last one, -1.  They are written to pool[r, :].
 *   block_table[b, k] = pool[r, k] for k < ceil(kv_len[b] / 128), -1 behind
 *   cu_pages[b + 1] = pages that requests 0..b took
 *   positions[t] = c + i,  slots[t] = page * 128 + positions[t] % 128 for the
 *     request's i-th new token t, -1 where no page is; rows behind the last
 *     token get 0 and -1
 *   free_out[0] = free pages that are left, free_out[1] = pages that were missing
 *
 * new_tokens, ctx_len  device int32 [batch].
 * rows         device int32 [batch], distinct, or NULL: request b has row b.  A
 *              row outside [0, pool_rows) holds no pages and takes none.
 * pool         device int32 [pool_rows, pool_blocks]: the pages of every request
 *              that the server holds; row r's first ceil(ctx_len / 128) entries are
 *              read.
 * free_pages   device int32 [free_size], of which the first free_count[0] are free
 *              (cut to [0, free_size]).  Pages that requests give back are written
 *              behind them by the caller, who raises the count.
 * free_count   device int32 [2] (the second is not read).
 * free_out     device int32 [2]; may be free_count itself (one small launch more).
 * max_blocks   blocks of a request that exist, 1..min(pool_blocks, 2^24): later ones get no
 *              page, and their tokens no slot.
 * T            rows of positions and slots: at least the sum of new_tokens.  (Where
 *              the sum is larger, nothing is written past T and cu_seqlens_q ends at
 *              T, but kv_len and the pages count all tokens: such a step's tables are
 *              not for use.)
 * block_size   128, as for msa_index_score.
 * cu_seqlens_q, cu_pages   device int32 [batch + 1], written in full, as are
 * kv_len, start_loc        device int32 [batch],
 * block_table              device int32 [batch, max_blocks],
 * positions, slots         device int32 and int64 [T].  (They and cu_pages are for the
 *                          caller's own kernels and books: no entry point here takes
 *                          them.)
 *
 * All arrays are compact; nothing that is written may overlap anything else
 * (MSA_ERR_STRIDE; but free_out and free_count).  Nothing is allocated or kept; a
 * call may be captured into a graph.  MSA_ERR_SHAPE for sizes out of range (batch
 * > 2^20, T, pool_rows, pool_blocks or free_size > 2^31 - 1, a pool of more than
 * 2^60 entries), MSA_ERR_NULL for a pointer that the call must use, MSA_ERR_HIP if a
 * launch fails.
 */
msa_status_t msa_step_tables(const int32_t* new_tokens, const int32_t* ctx_len,
                             const int32_t* rows, int32_t batch, int32_t* pool, int64_t pool_rows,
                             int64_t pool_blocks, const int32_t* free_pages, int64_t free_size,
                             const int32_t* free_count, int32_t* free_out, int64_t max_blocks,
                             int64_t T, int32_t block_size, int32_t* cu_seqlens_q, int32_t* kv_len,
                             int32_t* start_loc, int32_t* block_table, int32_t* positions,
                             int64_t* slots, int32_t* cu_pages, void* stream);

/* Output width RoundUp(max(max_blocks, 1), 16) (guide, section 五: the last
 * axis is aligned to 16, and an all-empty packed batch clamps MB to 1). */
int64_t msa_index_score_out_width(int64_t max_blocks);

/* A static, human-readable name for a status code. */
const char* msa_status_str(int32_t status);

/* Which kernel family a call with these sizes would use: 0 = decode tiles
 * (16 query rows per tile, for short query runs per request), 1 = prefill
 * tiles (hundreds of query rows per tile), chosen when requests average at
 * least 128 query rows (tokens times heads per KV group) and the batch has
 * at least 1024 (T * Hq).  Host-only; for benchmarks and tests. */
int32_t msa_index_score_kernel_family(int64_t T, int32_t batch, int32_t Hq, int32_t Hkv);

#ifdef __cplusplus
}
#endif

#endif /* MSA_INDEX_SCORE_H */
