/*
 * spec_verify_serve.h -- the paged serving operators around the verify step.
 *
 * One speculative decoding step of a server with a paged key/value cache is
 *   1. spec_verify_sample     the drafter's tokens from its logits, every row
 *                             with its own settings,
 *   2. spec_verify_slots      the cache pages of the new tokens (block tables
 *                             kept on the device) and each token's slot,
 *   3. spec_verify_append     the new keys and values into their slots (once
 *                             per layer),
 *   4. spec_verify_attention  every new token over its request's pages, the
 *                             block itself causally (once per layer),
 *   5. spec_verify            (spec_verify.h) the accepted tokens.
 * With rotary positions or a cache held in 8 bits, spec_verify_rope_append takes the
 * place of 3, and spec_verify_attention_ext reads that cache.  Where the drafter gives
 * a tree instead of a block,
 *      spec_verify_tree         forms masks and positions from the tree's parents
 *                               (after 2),
 *      spec_verify_attention_ext attends under the masks, and in place of 5 a token is
 *                               sampled from the target's logits at every row,
 *      spec_verify_tree_accept  finds the path that those tokens follow, and
 *      spec_verify_tree_move    moves its keys and values together (all layers).
 * None of these reads a length on the host, so a step can be enqueued
 * while the one before it still runs, and captured into a CUDA graph.
 *
 * Ownership, streams and errors are as in spec_verify.h: the caller owns
 * every buffer, calls only enqueue work on `stream`, argument errors come
 * back as SV_ERR_* before anything is enqueued, and data-dependent problems
 * are OR-ed into *dev_error (may be NULL; the caller zeroes it).  dtype is
 * SV_BF16 or SV_FP32; a cache may be SV_E4M3 where cache_dtype says so.  Strides are in elements; the last dimension is
 * contiguous.  Offsets are formed in 64 bits.
 */
#ifndef SPEC_VERIFY_SERVE_H
#define SPEC_VERIFY_SERVE_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* device error bits, next to those of spec_verify.h */
#define SV_DEVERR_PARAM 16  /* a row's sampling setting or random number is out of range */
#define SV_DEVERR_BLOCKS 32 /* the free list ran out of pages */
#define SV_DEVERR_PAGE 64   /* a page id or a slot lies outside the cache */

#define SV_DEVERR_TREE 128  /* a parent or a path that is not one of a tree */

/* cache_dtype besides SV_BF16 and SV_FP32: e4m3 codes (4 exponent bits, 3 mantissa bits,
 * no infinity, NaN 0x7f) and a power of two for each token and head: code * 2^exp. */
#define SV_E4M3 2

/* limits */
#define SV_SAMPLE_MAX_ROW_BYTES 1572864 /* V * element size of spec_verify_sample */
#define SV_SLOTS_MAX_B 8192             /* requests of one spec_verify_slots call */
#define SV_ATTN_MAX_HEAD_DIM 256        /* head_dim of spec_verify_attention */

/*
 * One token per row from processed logits and a given random number.
 *
 * For a row x with temperature T > 0: p = softmax(x / T), ranked by (value
 * desc, id asc) with -0 and +0 one value (the order of spec_verify); then
 * top_k keeps the k best, top_p the shortest prefix of those whose mass
 * reaches top_p of theirs, min_p drops what is below min_p times the largest
 * probability.  Of the kept set's mass Z the token is the smallest id whose
 * running mass over ascending ids exceeds u * Z (strictly).  T = 0: the
 * lowest id with the largest logit, with probability 1.  -inf is a mask.
 *
 *  logits       [N] rows of V, dtype; element aligned, row r at r * row_stride.
 *  row_stride   >= V.
 *  temperature  [N] float32 device, finite and >= 0, or NULL for 1.
 *  top_k        [N] int32 device or NULL; <= 0 or >= V is off.
 *  top_p        [N] float32 device in (0, 1] or NULL; 1 is off.
 *  min_p        [N] float32 device in [0, 1] or NULL; 0 is off.
 *  uniforms     [N] float32 device in [0, 1).
 *  out_tokens   [N] int32 device.
 *  out_probs    [N] float32 device or NULL: the token's probability in the
 *               kept set, renormalised.
 * A row with NaN or +inf or nothing but -inf (SV_DEVERR_NAN), or with a
 * setting out of range (SV_DEVERR_PARAM), gets token -1 and probability 0.
 * SV_ERR_UNSUPPORTED when V * element size exceeds SV_SAMPLE_MAX_ROW_BYTES.
 */
int spec_verify_sample(const void* logits, int64_t row_stride, int32_t N, int32_t V,
                       int32_t dtype, const float* temperature, const int32_t* top_k,
                       const float* top_p, const float* min_p, const float* uniforms,
                       int32_t* out_tokens, float* out_probs, int32_t* dev_error, void* stream);

/*
 * Block tables and slot maps of one step.  Request r has context_lens[r]
 * tokens in the cache, gets verify_lens[r] >= 0 new ones and holds the pages
 * block_table[r][0 .. held[r]).  After the call it holds exactly
 * need = ceil((context + new) / page_size) pages: pages above need go back to
 * the free list (requests in order, pages in order, pushed at free_count),
 * then missing ones are popped (requests in order, from the top of the list).
 * A finished request with context and new 0 gives everything back.
 *
 *  block_table     [B][table_stride >= width] int32 device, in place: entries
 *                  held .. need are written, no other one.
 *  held            [B] int32 device: pages held before the call.
 *  free_list       [free_cap] int32 device, in place: a stack of free page ids.
 *  free_count      [1] int32 device: ids on the stack before the call.
 *  n_rows          rows of positions and slots; at least the sum of verify_lens.
 *  out_row_offsets [B+1] int32: prefix sums of verify_lens.
 *  out_seq_lens    [B] int32: context + new; -1 for a request that is not served
 *                  or out of range (below).
 *  out_positions   [n_rows] int32: position of every new token in its request;
 *                  0 in the rows past the last token.
 *  out_slots       [n_rows] int64: page * page_size + offset; -1 in those rows.
 *  out_held        [B] int32 and out_free_count [1] int32: the counts after the
 *                  call.
 * No result may overlap context_lens, verify_lens, held or free_count (the kernel
 * reads those throughout; SV_ERR_ARG): a caller keeps two arrays of each count
 * and takes them in turn.
 *
 * Requests are served in order while pages last (SV_DEVERR_BLOCKS): one that
 * is not keeps what it holds and its tokens past those pages get slot -1.  A
 * request with a negative length, more pages than width or a held count
 * outside [0, width] (SV_DEVERR_LEN) keeps its pages and its slots are -1;
 * a verify_lens outside [0, n_rows] counts as no rows.  The tables of both kinds
 * do not hold their tokens' pages (entries past the held ones may name pages of
 * other requests), so their out_seq_lens is -1, which spec_verify_attention
 * refuses for the request alone: the step may run on before the flags are read.
 */
int spec_verify_slots(const int32_t* context_lens, const int32_t* verify_lens, int32_t B,
                      int32_t page_size, int32_t* block_table, int64_t table_stride,
                      int32_t width, const int32_t* held, int32_t* free_list, int32_t free_cap,
                      const int32_t* free_count, int32_t n_rows, int32_t* out_row_offsets,
                      int32_t* out_seq_lens, int32_t* out_positions, int64_t* out_slots,
                      int32_t* out_held, int32_t* out_free_count, int32_t* dev_error,
                      void* stream);

/*
 * New keys and values into their slots.  Row i of key and value
 * ([n_rows][kv_heads][head_dim], any row and head strides) is copied to
 * position slots[i] % page_size of page slots[i] / page_size of the caches
 * ([num_blocks][page_size][kv_heads][head_dim], any strides of the first
 * three dimensions, the same for both caches).  A negative slot is skipped; one past the caches
 * raises SV_DEVERR_PAGE and is skipped.  Where two rows have one slot, each of
 * its 2 to 16 byte units, keys and values apart, may be that of either.
 */
int spec_verify_append(const void* key, const void* value, int64_t k_row_stride,
                       int64_t k_head_stride, int64_t v_row_stride, int64_t v_head_stride,
                       const int64_t* slots, int32_t n_rows, int32_t kv_heads, int32_t head_dim,
                       void* key_cache, void* value_cache, int64_t block_stride,
                       int64_t token_stride, int64_t head_stride, int32_t num_blocks,
                       int32_t page_size, int32_t dtype, int32_t* dev_error, void* stream);

/*
 * Attention of a chunk of new tokens per request over its paged cache, which
 * already holds the new tokens' keys and values.
 *
 * Request r owns query rows row_offsets[r] .. row_offsets[r+1] - 1, l of them,
 * the last l of its seq_lens[r] tokens: row j has position p = seq - l + j and
 * sees the keys t with 0 <= t <= p and, with window > 0, t > p - window.  Query
 * head h reads key/value head h / (heads / kv_heads).
 *   out = sum_t softmax_t(scale q.k_t) v_t,   lse = log sum_t exp(scale q.k_t)
 * A row that sees no key (p < 0: l > seq) gets zeros and lse = -inf.  Keys and
 * values that a row does not see do not reach it, NaN and infinities included;
 * neither do page tails past seq_lens and table entries past the last page.
 *
 *  query        [n_rows][heads][head_dim]; strides multiples of 16 bytes.
 *  caches       as in spec_verify_append; base and strides multiples of 16 bytes.
 *  block_table  [B][table_stride >= table_width] int32 device.  A page id
 *               outside [0, num_blocks) raises SV_DEVERR_PAGE; a seq_len below 0
 *               or past table_width * page_size, or more rows than max_len, raise
 *               SV_DEVERR_LEN and the request's rows see no key; row_offsets that
 *               do not rise within [0, n_rows] raise it and the request's rows
 *               are not written.
 *  max_len      host upper bound of every l.
 *  n_rows       0 is no error: nothing is done.
 *  head_dim     a multiple of 8, up to SV_ATTN_MAX_HEAD_DIM; heads a multiple
 *               of kv_heads.  table_width * page_size up to 2^30 - 1, n_rows *
 *               heads up to 2^31 - 1 (SV_ERR_UNSUPPORTED).
 *  scale        factor of the scores, finite.
 *  window       <= 0: off.
 *  out          [n_rows][heads][head_dim] dtype, strides multiples of 16
 *               bytes; rows past row_offsets[B] are not written.
 *  out_lse      [n_rows][heads] float32 device or NULL.
 *  workspace    device scratch, 256-byte aligned, of at least
 *               spec_verify_attention_workspace_size bytes; needs no clearing.
 *               The size is that of all SMs' partials, whatever the call's (bf16
 *               heads of 128: 42 MB): a caller keeps one for all calls.
 *               Calls that share it must be ordered on the GPU.
 * bf16: scores and all sums are held in 32 bits, the weights exp(s - m) are
 * rounded to bf16 for the second product.  fp32: all in 32 bits.
 */
size_t spec_verify_attention_workspace_size(int32_t n_rows, int32_t heads, int32_t head_dim,
                                            int32_t dtype);
int spec_verify_attention(const void* query, int64_t q_row_stride, int64_t q_head_stride,
                          const void* key_cache, const void* value_cache, int64_t block_stride,
                          int64_t token_stride, int64_t head_stride, const int32_t* block_table,
                          int64_t table_stride, int32_t table_width, const int32_t* seq_lens,
                          const int32_t* row_offsets, int32_t B, int32_t n_rows, int32_t max_len,
                          int32_t heads, int32_t kv_heads, int32_t head_dim, int32_t num_blocks,
                          int32_t page_size, int32_t dtype, float scale, int32_t window,
                          void* out, int64_t o_row_stride, int64_t o_head_stride, float* out_lse,
                          int32_t* dev_error, void* workspace, size_t workspace_bytes,
                          void* stream);

/*
 * Rotary positions: the first rotary_dim dimensions of every head are pairs
 * (x, y), turned by the row's angle in the pair's plane,
 *   x' = amplitude (x cos - y sin),   y' = amplitude (y cos + x sin),
 * dimensions behind them are copied.  Pair i is dimensions (i, i + rotary_dim / 2), or
 * (2 i, 2 i + 1) where interleaved is not 0.  The angle is position * frequency:
 *
 *  positions    [n_rows] int32 device, any value.
 *  freqs        [rotary_dim / 2] int64 device: turns (of 2 pi) a position in units of
 *               2^-64, modulo 2^64, so that angles of far positions are exact.
 *  rotary_dim   even, 0 .. head_dim; 0 turns nothing and needs neither array.
 *  amplitude    finite factor of cos and sin.
 *  x, out       [n_rows][heads][head_dim] dtype, any row and head strides; out may be x
 *               itself (the same strides), or apart from it.
 * head_dim up to SV_ATTN_MAX_HEAD_DIM, n_rows * heads up to 2^30 - 1
 * (SV_ERR_UNSUPPORTED).  Products in fp32, rounded once.
 */
int spec_verify_rope(const void* x, int64_t row_stride, int64_t x_head_stride, int32_t n_rows,
                     int32_t heads, int32_t head_dim, int32_t dtype, const int32_t* positions,
                     const int64_t* freqs, int32_t rotary_dim, int32_t interleaved,
                     float amplitude, void* out, int64_t out_row_stride, int64_t out_head_stride,
                     void* stream);

/*
 * The same of queries and keys, with keys and values written into their slots of a
 * paged cache as by spec_verify_append (negative slots are skipped, ones past the
 * caches raise SV_DEVERR_PAGE; where two rows have one slot, what it holds is of
 * either, in parts).  heads 0: no queries; kv_heads 0: no keys and values.
 *
 *  query, out_query  [n_rows][heads][head_dim] dtype; out_query as `out` above.
 *  key, value        [n_rows][kv_heads][head_dim] dtype.
 *  caches            [num_blocks][page_size][kv_heads][head_dim] cache_dtype, any
 *                    strides of the first three dimensions, the same for both.
 *  cache_dtype       dtype, or SV_E4M3: a row of a head becomes codes and the smallest
 *                    exponent that brings its largest finite magnitude to 448 or below,
 *                    in [-100, 119] (magnitudes above 448 * 2^119 become that).  Codes
 *                    are rounded to the nearest, ties to even, from fp32; what is not
 *                    finite becomes NaN.
 *  key_exps, value_exps  [num_blocks][page_size][kv_heads] int8 device for SV_E4M3,
 *                    strides e_* in elements, the same for both; else not read.
 * n_rows * (heads + 2 * kv_heads) up to 2^30 - 1.  Any alignment of the elements; whole
 * 16-byte units, and head_dim and rotary_dim multiples of 8, are fastest.
 */
int spec_verify_rope_append(const void* query, int64_t q_row_stride, int64_t q_head_stride,
                            int32_t heads, const void* key, const void* value,
                            int64_t k_row_stride, int64_t k_head_stride, int64_t v_row_stride,
                            int64_t v_head_stride, int32_t kv_heads, int32_t n_rows,
                            int32_t head_dim, int32_t dtype, const int32_t* positions,
                            const int64_t* freqs, int32_t rotary_dim, int32_t interleaved,
                            float amplitude, void* out_query, int64_t oq_row_stride,
                            int64_t oq_head_stride, const int64_t* slots, void* key_cache,
                            void* value_cache, int64_t block_stride, int64_t token_stride,
                            int64_t head_stride, int32_t num_blocks, int32_t page_size,
                            int32_t cache_dtype, int8_t* key_exps, int8_t* value_exps,
                            int64_t e_block_stride, int64_t e_token_stride, int64_t e_head_stride,
                            int32_t* dev_error, void* stream);

/*
 * spec_verify_attention over a cache of 8 bits, of a tree of drafted tokens, or both.
 * What follows differs from it; the workspace is the same.
 *
 *  cache_dtype  dtype, or SV_E4M3 with dtype SV_BF16: codes (base and strides multiples
 *               of 16 bytes, head_dim a multiple of 16) and exponents as above, any int8.
 *               The strides of the exponents up to 2^31 - 1.
 *  tree_mask    [n_rows][mask_words] int32 device, or NULL: a block, causal.  Row j of a
 *               request of l rows sees its context's keys t < seq - l and, of its own rows'
 *               keys seq - l + i, those with i <= j whose bit i (bit i % 32 of word i / 32)
 *               is set.  A row that sees no key gets zeros and lse = -inf.  A seq_len
 *               below l raises SV_DEVERR_LEN and the request's rows see no key.
 *  mask_words   at least ceil(max_len / 32).
 *  positions    [n_rows] int32 device: for a tree with window > 0, else not read: row j
 *               sees the context's keys t > positions[row] - window (positions outside
 *               [seq - l, seq - 1] are brought there); of its own rows the mask decides.
 * Over codes, scores and sums are held in 32 bits and the weights are rounded to fp16:
 * 2^-11 of each, and of small ones 2^-32 of the row's largest, a weight counted with the
 * largest power of two 2^e of its tile's values: a key's part of the output is off by at
 * most 2^-32 448 w, w the row's largest softmax 2^e.  Keys and values are exact
 * but for rows far below the largest of their tile, the request's tokens 64 i .. 64 i + 63:
 * of rows whose exponent is more than 22 below the tile's largest (or below -102) up to
 * 2^-23 in units of 2^largest is lost.  Rows of the tile that a query does not see count
 * among them, and reach it in this way alone.  Of a query's row and head, elements below
 * 2^-31 of the largest may lose up to 2^-39 of it.
 */
int spec_verify_attention_ext(
    const void* query, int64_t q_row_stride, int64_t q_head_stride, const void* key_cache,
    const void* value_cache, int64_t block_stride, int64_t token_stride, int64_t head_stride,
    int32_t cache_dtype, const int8_t* key_exps, const int8_t* value_exps, int64_t e_block_stride,
    int64_t e_token_stride, int64_t e_head_stride, const int32_t* block_table,
    int64_t table_stride, int32_t table_width, const int32_t* seq_lens,
    const int32_t* row_offsets, const int32_t* tree_mask, int32_t mask_words,
    const int32_t* positions, int32_t B, int32_t n_rows, int32_t max_len, int32_t heads,
    int32_t kv_heads, int32_t head_dim, int32_t num_blocks, int32_t page_size, int32_t dtype,
    float scale, int32_t window, void* out, int64_t o_row_stride, int64_t o_head_stride,
    float* out_lse, int32_t* dev_error, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Masks and positions of a step's trees.  Request r's rows row_offsets[r] ..
 * row_offsets[r+1] - 1, l of them, are the last l of its seq_lens[r] tokens; row 0 is
 * the last accepted token, the others drafted ones, each after its parent.
 *
 *  parents       [n_rows] int32 device: the parent's number among the request's rows,
 *                below the row's own; -1: a root.  Others raise SV_DEVERR_TREE and the
 *                row counts as a root.
 *  max_len       host upper bound of every l, up to SV_MAX_LEN (SV_ERR_UNSUPPORTED).
 *  out_positions [n_rows] int32: seq - l + the steps up to the root.
 *  out_mask      [n_rows][mask_words] int32, mask_words >= ceil(max_len / 32): bits of
 *                the row itself and of all above it.
 * Rows past row_offsets[B], and those of a request with more rows than max_len or
 * tokens fewer than its rows (SV_DEVERR_LEN), get position 0 and an empty mask;
 * row_offsets that do not rise within [0, n_rows] raise SV_DEVERR_LEN too and the
 * request's rows are not written.
 */
int spec_verify_tree(const int32_t* parents, const int32_t* seq_lens, const int32_t* row_offsets,
                     int32_t B, int32_t n_rows, int32_t max_len, int32_t* out_positions,
                     int32_t* out_mask, int32_t mask_words, int32_t* dev_error, void* stream);

/*
 * The accepted path of every request's tree.  It starts at row 0; from a row it goes
 * on to that child whose token is the row's next token (of several the lowest), as long
 * as there is one; none follows a next token below 0, which spec_verify_sample gives
 * where it can draw none.  With next_tokens sampled from the target's rows
 * (spec_verify_sample) the tokens given out are distributed as the target's, whatever was
 * drafted.
 *
 *  tokens, next_tokens, parents  [n_rows] int32 device: each row's own token, the
 *                  target's after it, and the parents as above (ones out of range raise
 *                  SV_DEVERR_TREE; such rows, and roots other than row 0, are not
 *                  accepted).
 *  out_tokens      [n_rows] int32: a request's tokens of the step from its first row,
 *                  accept_len + 1 of them: the accepted drafts and the target's token
 *                  after the last; then -1.
 *  out_path        [n_rows] int32: the rows of the path, from its first row (row 0); then
 *                  -1.
 *  out_accept_len  [B] int32: accepted drafts; -1 for a request without rows or out of
 *                  range (more rows than max_len, bad row_offsets: SV_DEVERR_LEN).
 * Rows past row_offsets[B] get -1.
 */
int spec_verify_tree_accept(const int32_t* tokens, const int32_t* next_tokens,
                            const int32_t* parents, const int32_t* row_offsets, int32_t B,
                            int32_t n_rows, int32_t max_len, int32_t* out_tokens,
                            int32_t* out_path, int32_t* out_accept_len, int32_t* dev_error,
                            void* stream);

/*
 * Keys and values of the accepted paths, moved together: the cache row at slot
 * slots[row0 + path[row0 + j]] goes to slots[row0 + j] for 1 <= j <= accept_len[r], as
 * if all were read before any is written, in every layer; row 0 stays, wherever the path
 * starts.  A slot below 0 at either end
 * leaves that row out, one past the caches does and raises SV_DEVERR_PAGE.  A path that
 * does not rise, path[j] < j or path[j] >= l, ends there (SV_DEVERR_TREE); an accept_len
 * outside [-1, l - 1] raises SV_DEVERR_LEN and moves nothing of the request.
 *
 *  slots        [n_rows] int64 device, as spec_verify_slots gives them.
 *  caches       [layers][num_blocks][page_size][kv_heads][head_dim] cache_dtype, any
 *               strides of the first four dimensions, the same for both.
 *  key_exps, value_exps  [layers][num_blocks][page_size][kv_heads] int8 for SV_E4M3.
 */
int spec_verify_tree_move(const int32_t* path, const int32_t* accept_len,
                          const int32_t* row_offsets, const int64_t* slots, int32_t B,
                          int32_t n_rows, int32_t max_len, int32_t layers, int32_t kv_heads,
                          int32_t head_dim, void* key_cache, void* value_cache,
                          int64_t layer_stride, int64_t block_stride, int64_t token_stride,
                          int64_t head_stride, int32_t num_blocks, int32_t page_size,
                          int32_t cache_dtype, int8_t* key_exps, int8_t* value_exps,
                          int64_t e_layer_stride, int64_t e_block_stride, int64_t e_token_stride,
                          int64_t e_head_stride, int32_t* dev_error, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_VERIFY_SERVE_H */
