/*
 * attn_packed.h - steps that add several tokens per request over the paged cache
 * of attn_paged.h: prompts (or chunks of them) of different lengths packed into
 * one call, and trees of drafted tokens with what plans and commits them.
 *
 * A step runs: attn_page_plan hands out pages and slots for the new tokens,
 * attn_kv_append_paged writes their keys and values, and attn_prefill_paged
 * attends them; a step of drafted tokens has attn_draft_plan behind the page plan
 * (whose positions the append then takes), attn_decode_tree in every layer, and
 * attn_draft_commit once the accepted path is known.
 *
 * Conventions, types, error codes and the cache's layout and limits are those of
 * attn.h and attn_paged.h.  In addition:
 *
 *  - New tokens are packed: cu_new is DEVICE int32 [B + 1], 0 first and rising (what
 *    attn_page_plan writes); request b has n_b = cu_new[b + 1] - cu_new[b] new tokens,
 *    token i in row cu_new[b] + i of the packed arrays.  Rows at or behind their end
 *    (T) do not exist.  Other contents of cu_new give rows without meaning, but
 *    nothing outside the arrays is touched.
 *  - The new tokens are in the cache already, as the last n_b of the request's
 *    L = seqlens[b] tokens: token i is at place L - n_b + i.  L is clamped to
 *    0 .. max_blocks * page_size.
 *  - T * n_h < 2^31 (else ATTN_ERR_ARG).
 *  - No array may overlap an output (ATTN_ERR_ARG where the sizes tell).
 */
#ifndef ATTN_PACKED_H
#define ATTN_PACKED_H

#include "attn_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * attn_packed_workspace_size - bytes of device scratch that attn_prefill_paged and
 * attn_decode_tree need for these sizes; -1 cast to size_t for invalid ones.  The
 * caller owns it; calls that may overlap on the GPU (other streams, captured graphs)
 * need one each.
 */
ATTN_API size_t attn_packed_workspace_size(int T, int B, int n_h, int n_kv, int D_qk, int D_v, int page_size,
                                           int max_blocks, attn_dtype_t dtype);

/*
 * attn_prefill_paged - causal attention of packed new tokens over a paged cache: the
 * token at place p attends tokens 0 .. p of its request through row b of block_table.
 * Whole prompts (L = n_b), chunks behind what the cache holds (L > n_b) and single
 * tokens (n_b = 1, attn_decode_paged's step) may be mixed in one call.
 *
 *   q, out     [T, n_h, D_qk] (un-rotated) and [T, n_h, D_v].
 *   positions  DEVICE int32 [T] or NULL: the position at which a row's query is
 *              rotated (NULL: its place).  A negative one marks an empty row, as
 *              attn_page_plan does for refused requests.
 *   lse        fp32 [T, n_h] or NULL: natural-log log-sum-exp of the row's scaled scores.
 *   v_token_stride and the other arguments as in attn_decode_paged.
 * Rows that are empty, that see no key (a place below 0) or that lie behind
 * cu_new[B] come out as 0, their lse as -inf.
 *
 * bf16 with D_qk = D_v = 64 or 128, at most 128 query heads per KV head and a RoPE
 * span of whole 16-byte pieces (none, or rope_offset % 8 == 0 and rope_dims % 8 == 0,
 * % 16 with ATTN_ROPE_HALF) runs on the tensor cores, anything else on CUDA cores.
 * Sums are fp32.  On the tensor cores softmax weights are rounded to bf16 on the way in,
 * and so are rotated queries (their sines are off by 2^-21).  With RoPE, what that leaves
 * of 64 of the query's dims and, with D = 128, of half of the weights is kept; without it
 * queries go in as they are.  Either way an output's error is about 1.45 times that of
 * its own rounding (for normally distributed inputs).
 * NaN or an infinity in a query, key or value reaches the rows that see it and no
 * other: values at places that a row does not see, of other requests or behind the last
 * token may be anything.  A key with a score of -inf has no weight, a row whose scores
 * all are comes out as one that sees no key, and a score of +inf makes its row NaN.  An
 * infinite value gives its dim of the rows that see it that infinity, or NaN where the
 * key's weight is 0 (one below 2^-110 of the row's largest may count as 0).
 * The workspace of shapes that the tensor cores take holds T * n_h * (D + 64) * 2 bytes
 * for the rotated queries, beside the partials of the pieces that requests are cut into.
 * Outputs must not overlap inputs, the workspace or each other.
 */
ATTN_API int attn_prefill_paged(const void* q, const void* k_pages, const void* v_pages, int v_token_stride,
                                const int* block_table, const int* cu_new, const int* seqlens, const int* positions,
                                void* out, float* lse, int T, int B, int n_h, int n_kv, int D_qk, int D_v,
                                int n_pages, int page_size, int max_blocks, float rope_base, int rope_offset,
                                int rope_dims, float scale, attn_dtype_t dtype, void* workspace,
                                size_t workspace_bytes, void* stream);

/*
 * attn_decode_tree - attention of drafted tokens that form a tree (or any set with
 * its own visibility): drafted token i of request b sees the L - n_b tokens in front
 * of the drafts and those drafted tokens j whose bit is set in its row of `visible`.
 *
 *   visible    DEVICE int32 [T, words], 1 <= words <= 4 (else ATTN_ERR_ARG): bit j % 32
 *              of word j / 32 of row cu_new[b] + i stands for drafted token j of the
 *              same request.  Bits of tokens that the request does not have are
 *              ignored; drafted tokens at or behind 32 * words are seen by none.
 *              The token itself is seen when its own bit says so.
 *   positions  as in attn_prefill_paged; a drafted token's is the number of tokens in
 *              front of the drafts plus its depth (attn_draft_plan).
 * Everything else as attn_prefill_paged.
 */
ATTN_API int attn_decode_tree(const void* q, const void* k_pages, const void* v_pages, int v_token_stride,
                              const int* block_table, const int* cu_new, const int* seqlens, const int* positions,
                              const int* visible, int words, void* out, float* lse, int T, int B, int n_h, int n_kv,
                              int D_qk, int D_v, int n_pages, int page_size, int max_blocks, float rope_base,
                              int rope_offset, int rope_dims, float scale, attn_dtype_t dtype, void* workspace,
                              size_t workspace_bytes, void* stream);

/*
 * attn_draft_plan - positions and visibility of drafted tokens from their parents.
 *
 *   parents    DEVICE int32 [T]: the parent of drafted token i of a request, as an index
 *              0 .. i - 1 among the same request's drafts, or -1 for a root (a child of
 *              the last token in front of the drafts).  Several roots are fine.
 *   places     DEVICE int32 [T]: the tokens' places, as attn_page_plan's positions; a
 *              negative one marks an empty row.
 *   positions  [T]: places[t] - i + depth(i), depth 0 for a root and one more than the
 *              parent's otherwise.
 *   visible    [T, words], 1 <= words <= 4 (else ATTN_ERR_ARG): the bits of the token's
 *              ancestors and its own.
 * A token with a parent outside -1 .. i - 1, at or behind 32 * words, or with such an
 * ancestor, as well as an empty row and rows behind cu_new[B], gets position -1 and no
 * bit.  Outputs must not overlap inputs or each other.  One kernel.
 */
ATTN_API int attn_draft_plan(const int* places, const int* cu_new, const int* parents, int* positions, int* visible,
                             int T, int B, int words, void* stream);

/*
 * attn_draft_commit - the accepted drafts of each request move to consecutive places
 * behind the tokens it held, and pages that the rest leaves go back on the stack.
 *
 *   lens     DEVICE int32 [B]: tokens in front of the drafts (below 0: 0).
 *   seqlens  DEVICE int32 [B]: tokens with all drafts (clamped as above).
 *   path     DEVICE int32 [B, max_path], 1 <= max_path <= 128 (else ATTN_ERR_UNSUPPORTED):
 *            the accepted drafts of request b are path[b][0] .. path[b][n_path[b] - 1],
 *            rising.  The path ends early in front of an index that does not rise, is
 *            negative or has lens[b] + index >= seqlens[b]; a_b tokens remain.
 *   token at place lens[b] + path[b][i]  ->  place lens[b] + i, for i < a_b
 *   new_lens[b] = lens[b] + a_b
 *   v_pages  NULL: values alias the keys (MLA).  v_token_stride as in attn_decode_paged.
 *   free_pages [free_cap], n_free [1], n_left [1]: the stack of attn_page_plan, or all
 *            NULL to leave the pages with their requests.  The pages
 *            ceil(new_lens[b] / page_size) .. ceil(seqlens[b] / page_size) - 1 of each
 *            row are put on its top, request after request, in rising order, but for
 *            entries outside [0, n_pages), which are no pages (a row is as long as
 *            seqlens says); n_left is its height after that, at most free_cap (pages
 *            behind it are dropped).
 *            The table keeps its entries.  Called twice with the same n_free, the second
 *            call puts the same pages in the same places.
 * A token with its old or new page outside [0, n_pages) is not moved.  Pages are owned
 * by one request each as far as they are written here.  Outputs must not overlap inputs
 * or each other.  B <= 16384 (else ATTN_ERR_UNSUPPORTED).  One kernel.
 */
ATTN_API int attn_draft_commit(void* k_pages, void* v_pages, int v_token_stride, const int* block_table,
                               const int* lens, const int* seqlens, const int* path, const int* n_path,
                               int* new_lens, int* free_pages, const int* n_free, int* n_left, int B, int max_path,
                               int n_kv, int D_qk, int D_v, int n_pages, int page_size, int max_blocks, int free_cap,
                               attn_dtype_t dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_PACKED_H */
