/*
 * attn_paged.h - the paged-cache part of libattn.so's C ABI: a KV cache whose
 * tokens live in pages that any request may own, the plan that hands the pages
 * out, the append that writes new tokens into them, and single-token decode
 * over them - alone, or for a batch whose requests start with the same pages.
 *
 * The KV cache decides how many requests one card holds ("Transformer 与 LLM"
 * slide 06); pages keep only the tokens that exist, and tokens that several
 * requests share are kept once.  Conventions, types and error codes are those
 * of attn.h.  In addition:
 *
 *  - A cache is k_pages [n_pages, page_size, n_kv, D_qk] and v_pages
 *    [n_pages, page_size, n_kv, D_v]: slot s = page * page_size + row holds one
 *    token.  page_size is a power of two from 16 to 256 (else
 *    ATTN_ERR_UNSUPPORTED) and n_pages * page_size < 2^31 (else ATTN_ERR_ARG).
 *  - block_table is DEVICE int32 [B, max_blocks]: entry (b, j) is the page that
 *    holds tokens j * page_size .. of request b.  Entries behind a request's
 *    last token are never read.  max_blocks * page_size <= 2^31 - 2^16
 *    (else ATTN_ERR_ARG).
 *  - A page index outside [0, n_pages) in front of a request's last token reads
 *    as keys and values of zero; nothing outside the cache is read or written.
 *  - Tokens are rotated at any 32-bit position, with angles to some 1e-6 rad and
 *    |position| * 2^-48 more (1e-5 rad at 2^31).
 *  - int32 pointers are 4-byte aligned, all others 16-byte (ATTN_ERR_ALIGN).
 *  - Results do not depend on the order in which blocks of a kernel run: the
 *    same call on the same inputs gives the same bits.
 */
#ifndef ATTN_PAGED_H
#define ATTN_PAGED_H

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * attn_page_plan - block tables, slots and positions of one step's new tokens,
 * from the requests' lengths.  Request b holds lens[b] tokens and adds
 * n_new[b] (values below 0 count as 0); the new tokens of all requests are
 * packed one request after the other, request b's first being row cu_new[b].
 *
 *   cu_new[b]  = sum of n_new over the requests before b (cu_new[B]: of all)
 *   need(b)    = ceil((lens[b] + n_new[b]) / page_size) - ceil(lens[b] / page_size)
 *   its pages  = free_pages[n_free - 1 - off], off from sum of need over the
 *                requests before b, in rising order: the free pages are a stack
 *                and the plan takes them from its top
 *   slots[cu_new[b] + i]     = page of token lens[b] + i, times page_size, plus
 *                              the token's row in that page
 *   positions[cu_new[b] + i] = lens[b] + i
 *   seqlens[b] = lens[b] + n_new[b]
 *
 * A request is refused - its table row stays as it is, its tokens get slot and
 * position -1, seqlens[b] = lens[b] - when lens[b] + n_new[b] tokens pass
 * max_blocks pages, when its rows pass max_tokens, or when it needs pages and
 * the stack does not reach that far (requests refused for the first two
 * reasons need no pages; one refused for the third leaves the stack's rest to
 * nobody, so that the requests behind it that need pages are refused too).
 *
 *   lens, n_new  DEVICE int32 [B].
 *   block_table  [B, max_blocks]: the entries of newly taken pages are written,
 *                the entry of each request's partly filled last page is read.
 *   free_pages   DEVICE int32 [free_cap]; n_free DEVICE int32 [1]: pages on the
 *                stack (clamped to 0 .. free_cap).  free_cap <= n_pages (else
 *                ATTN_ERR_ARG).
 *   seqlens [B], cu_new [B + 1], slots and positions [max_tokens], n_left [1]:
 *                outputs, int32.  Rows behind the last new token get -1.
 *                n_left is the stack's height after the step; a released page is
 *                put back by writing it on top.  Sums past 2^31 - 1 saturate.
 * A page index outside [0, n_pages) in the stack or the table gives slot -1.
 * Outputs must not overlap inputs or each other (ATTN_ERR_ARG).  B <= 16384
 * (else ATTN_ERR_UNSUPPORTED).  One kernel.
 */
ATTN_API int attn_page_plan(const int* lens, const int* n_new, int* block_table, const int* free_pages,
                            const int* n_free, int* seqlens, int* cu_new, int* slots, int* positions, int* n_left,
                            int B, int max_blocks, int page_size, int n_pages, int free_cap, int max_tokens,
                            void* stream);

/*
 * attn_kv_append_paged - attn_kv_append into pages: row t of k_new is rotated at
 * positions[t] (the cache keeps rotated keys, "Transformer架构完全深度解析" §7)
 * and stored at slots[t], its value row is copied there.  Rows whose slot lies
 * outside [0, n_pages * page_size) are skipped.
 *
 *   k_new   [T, n_kv, D_qk]; v_new [T, n_kv, D_v], or NULL when values alias the
 *           keys (MLA), which v_pages must not overlap otherwise (ATTN_ERR_ARG);
 *           v_token_stride as in attn_decode (0 = n_kv * D_v).
 *   slots   DEVICE int32 [T]; slots of one call must differ (of two rows with the
 *           same slot either may be stored, mixed in pieces of 8 dims).
 *   positions DEVICE int32 [T]; may be NULL when rope_base <= 0.
 * Other arguments and their limits as attn_kv_append.
 */
ATTN_API int attn_kv_append_paged(const void* k_new, const void* v_new, void* k_pages, void* v_pages,
                                  int v_token_stride, const int* slots, const int* positions, int T, int n_kv,
                                  int D_qk, int D_v, int n_pages, int page_size, float rope_base, int rope_offset,
                                  int rope_dims, attn_dtype_t dtype, void* stream);

/*
 * attn_decode_paged_workspace_size - bytes of device scratch that
 * attn_decode_paged (prefix_len = 0) and attn_decode_shared need for these
 * sizes; -1 cast to size_t for invalid ones.  It grows with the rows B * n_h, not
 * with max_blocks.  The caller owns it; calls that may overlap on the GPU (other
 * streams, captured graphs) need one each.
 */
ATTN_API size_t attn_decode_paged_workspace_size(int B, int n_h, int n_kv, int D_qk, int D_v, int page_size,
                                                 int max_blocks, int prefix_len, attn_dtype_t dtype);

/*
 * attn_decode_paged - attn_decode over a paged cache: the new token of request b
 * at position seqlens[b] - 1 attends tokens 0 .. seqlens[b] - 1 through row b of
 * block_table.
 *
 *   seqlens  DEVICE int32 [B], the new token included.  seqlens[b] <= 0 marks an
 *            empty place of a padded batch: its output row is 0 and its lse
 *            -inf.  Values above max_blocks * page_size are clamped to it.
 *   v_token_stride  elements between consecutive slots of v_pages (0: n_kv * D_v);
 *            MLA passes v_pages = k_pages and v_token_stride = D_qk.
 * Outputs must not overlap inputs, the workspace or each other.
 * Other arguments, sizes and errors as attn_decode.  On the tensor cores run bf16 with
 * D_qk = D_v = 64 or 128, at most 128 query heads per KV head and RoPE over the whole
 * head or none, and the MLA-absorbed shape (128 heads over one of 576 dims, v_pages =
 * k_pages); other shapes on CUDA cores.  Sums are fp32; queries after RoPE and softmax
 * weights are rounded to bf16 on the way into the tensor cores, but for pieces of at
 * most 64 rows (a request's own keys under up to 64 heads per KV head, the shared
 * prefix of a small batch), which keep what that rounding leaves: an output's error is
 * then that of its own rounding, else larger (1.3 times without RoPE, 1.7 with it, for
 * normally distributed inputs).  NaN in a query, key or
 * value reaches the rows that see it and no other; an infinite value gives them that
 * infinity (both infinities in one dim, or a weight of 0: NaN); a key with a score of -inf
 * has no weight, one with a score of inf makes its rows NaN.
 */
ATTN_API int attn_decode_paged(const void* q, const void* k_pages, const void* v_pages, int v_token_stride,
                               const int* block_table, const int* seqlens, void* out, float* lse, int B, int n_h,
                               int n_kv, int D_qk, int D_v, int n_pages, int page_size, int max_blocks,
                               float rope_base, int rope_offset, int rope_dims, float scale, attn_dtype_t dtype,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * attn_decode_shared - attn_decode_paged for a batch whose requests all start
 * with the same prefix_len tokens (a system prompt, a document): the prefix is
 * read and multiplied once for the whole batch - one product of the B * n_h / n_kv
 * query rows of each KV head with its prefix keys - and joined with each
 * request's own keys by the log-sum-exp rule ("Transformer架构完全深度解析" §13).
 * The MLA-absorbed shape on the tensor cores is the exception: the prefix is kept
 * once, but read (from L2) and multiplied for each request, so that a call costs
 * as much as attn_decode_paged over the same lengths.
 *
 *   prefix_pages  DEVICE int32 [prefix_len / page_size]: the pages of the prefix
 *            (what every row of block_table starts with; those entries of
 *            block_table are not read).
 *   prefix_len  > 0, whole pages (a multiple of page_size) and at most
 *            max_blocks * page_size, else ATTN_ERR_ARG.
 *   seqlens  the prefix included: request b has seqlens[b] - prefix_len tokens of
 *            its own, at least its new one.  seqlens[b] <= prefix_len marks an
 *            empty place of a padded batch (output row 0, lse -inf).
 * Everything else as attn_decode_paged, whose result it equals up to rounding.
 */
ATTN_API int attn_decode_shared(const void* q, const void* k_pages, const void* v_pages, int v_token_stride,
                                const int* prefix_pages, int prefix_len, const int* block_table, const int* seqlens,
                                void* out, float* lse, int B, int n_h, int n_kv, int D_qk, int D_v, int n_pages,
                                int page_size, int max_blocks, float rope_base, int rope_offset, int rope_dims,
                                float scale, attn_dtype_t dtype, void* workspace, size_t workspace_bytes,
                                void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_PAGED_H */
