/*
 * dsa_paged.h — C ABI of the paged key-value cache that follows the indexer.
 *
 * The indexer (dsa_index.h) answers which key positions attention should
 * read.  The calls here keep the keys and values those positions name and
 * read them: page tables and slot maps from request lengths, the cache write,
 * and attention of new queries over all cached tokens or over the positions
 * the indexer chose (MLI — Core Idea: the selected k positions are what
 * sparse attention computes over; PIVOT abstract: prefill and decode).
 *
 * A cache is a pool of pages.  K and V are [n_pages, page, Hkv, d]; the three
 * inner dimensions are contiguous, pages lie `page_stride` elements apart
 * (page_stride >= page * Hkv * d, so K and V may share one buffer side by
 * side).  Token `pos` of request b lives in page block_table[b, pos / page],
 * at offset pos % page; its slot number is page_id * page + offset.  e4m3
 * pages come with fp32 scales [n_pages, page, Hkv] (contiguous): the value of
 * an element is e4m3(byte) * scale[page, offset, head].
 *
 * Conventions are those of dsa_index.h: device pointers on the current
 * device, contiguous unless a stride is named; outputs overlap inputs only
 * where a call says so.  Q, k, v, out and the workspace are 16-byte aligned,
 * all else to its element (pages on 16 bytes are written and read faster);
 * other pointers are refused (DSA_ERR_INVALID_ARG).  The caller
 * owns every buffer; the first bytes of the workspace hold the status word
 * (zero its first 8 bytes before its first use, read it with
 * dsa_check_status); calls are asynchronous on `stream`, allocate nothing and
 * can be captured into a CUDA graph.  A workspace serves one call at a time.
 * Queries, keys and values must be finite in every slot below a request's
 * length, values below 2^80 in magnitude (sums are kept unnormalised); slots at
 * or beyond it may hold anything.
 */
#ifndef DSA_PAGED_H
#define DSA_PAGED_H

#include "dsa_index.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Page plan: block tables and slot maps of one step, from request lengths.
 *   lens [B], new_lens [B] int32: tokens each request holds, and the tokens
 *          this step adds to it (either may be 0)
 *   free_pages [n_free] int32: page ids not in use, handed out in order;
 *   used [1] int32 (device): how many of them are handed out already
 *   block_table [B, max_pages] int32, in and out: request b's first
 *          ceil(lens[b] / page) entries are read, the entries up to
 *          ceil((lens[b] + new_lens[b]) / page) are written with new pages
 *          (request after request, in order), all others stay as they were
 *   q_offsets [B+1] int32: exclusive sum of new_lens
 *   slots [max_tokens] int64, positions [max_tokens] int32: slot and position
 *          of each new token, request after request; -1 behind the last one
 *   lens_out [B] int32 = lens + new_lens (may be `lens` itself)
 *   used_out [1] int32 = used + pages handed out (may be `used` itself)
 * Checked on the device, before anything is handed out: lengths >= 0,
 * lens + new_lens <= max_pages * page, sum of new_lens <= max_tokens,
 * 0 <= used <= n_free (else DSA_ERR_INVALID_ARG in the status word), enough
 * free pages (else DSA_ERR_PAGES).  A step that fails leaves block_table as
 * it was and answers with no tokens: q_offsets 0, slots and positions -1,
 * lens_out = lens, used_out = used.  A page id outside 0 .. n_pages - 1 is
 * recorded as DSA_ERR_INVALID_ARG; the slots in it are -1.
 * B = 0 is an empty call: nothing is launched and every output stays as it
 * was.  B <= 2^20, max_pages * page < 2^31.
 * ---------------------------------------------------------------------- */
int dsa_page_plan_workspace_size(int B, int max_tokens, size_t* bytes);
int dsa_page_plan(const int32_t* lens, const int32_t* new_lens, const int32_t* free_pages, int n_free,
                  const int32_t* used, int B, int page, int n_pages, int max_pages, int max_tokens,
                  int32_t* block_table, int32_t* q_offsets, int64_t* slots, int32_t* positions,
                  int32_t* lens_out, int32_t* used_out, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Cache write: rows k, v [T, Hkv, d] go to the slots the plan named.
 *   slots [T] int64: a negative slot skips its row; a slot beyond the pool
 *          skips it and records DSA_ERR_INVALID_ARG.  Slots must be distinct:
 *          rows that name the same one leave it unspecified.
 *   v, V   may both be NULL (a cache of keys alone, such as the indexer's)
 *   src_dtype bf16 or fp32; kv_dtype the same, or e4m3, which stores
 *          scale = max(amax over d / 448, 2^-126) in K_scale / V_scale and
 *          e4m3(x / scale), rounded to nearest even.  A row and head that
 *          holds an infinity or a NaN gets a scale of NaN, and reads back so.
 *   d <= 256.  T = 0 is an empty call.  The workspace needs 256 bytes.
 * ---------------------------------------------------------------------- */
int dsa_page_append(const void* k, const void* v, const int64_t* slots, int T, int Hkv, int d, int src_dtype,
                    int kv_dtype, void* K, void* V, float* K_scale, float* V_scale, int n_pages, int page,
                    int64_t page_stride, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Attention of new queries over all cached tokens.
 *   Q [total_q, Hq, d] bf16 or fp32; out the same shape and type
 *   q_offsets [B+1] int32: request b owns rows q_offsets[b] ..
 *          q_offsets[b+1] - 1 (m_b of them, 0 <= m_b <= max_q); rows in front
 *          of q_offsets[0] and from q_offsets[B] on belong to none: their
 *          outputs stay as they were
 *   lens [B] int32: tokens of request b, its new ones included
 *   Query row j of request b sits at position lens[b] - m_b + j and sees the
 *   tokens up to and including it; head h reads key head h / (Hq / Hkv):
 *       out[j, h] = sum_s p_s v_s,  p = softmax_s(scale * q[j, h] . k_s)
 *   A query that sees no token has out 0 and lse -inf.
 *   A NaN in a query row, or in a key or scale that it reads, shows in its
 *   outputs and lse; only an e4m3 NaN byte under a finite scale, which the
 *   cache write never leaves, may read as a number.
 *   softmax_scale: HOST pointer to the scale, NULL for d^-1/2
 *   lse [total_q, Hq] fp32: log sum_s exp(scale q . k_s), or NULL
 *   Checked on the device: 0 <= lens[b] <= max_pages * page, offsets that
 *   ascend within 0 .. total_q, m_b <= max_q, page ids within the pool.  A
 *   request that fails is skipped, nothing outside the pool is read, and
 *   either records DSA_ERR_INVALID_ARG (the outputs of such a call are
 *   unspecified).
 *   Hq a multiple of Hkv, Hq <= 1024, Hq / Hkv <= 128, d <= 256,
 *   1 <= max_q <= 65536, max_pages * page <= 2^31 - 1024.  fp32 queries
 *   take fp32 pages, bf16 queries bf16 or e4m3 pages.
 * Sums and softmax statistics are fp32.
 * ---------------------------------------------------------------------- */
int dsa_attend_paged_workspace_size(int B, int total_q, int max_q, int Hq, int Hkv, int d, int q_dtype,
                                    int kv_dtype, size_t* bytes);
int dsa_attend_paged(const void* Q, const void* K, const void* V, const float* K_scale, const float* V_scale,
                     const int32_t* block_table, const int32_t* lens, const int32_t* q_offsets, int B, int total_q,
                     int max_q, int n_pages, int page, int64_t page_stride, int max_pages, int Hq, int Hkv, int d,
                     const float* softmax_scale, int q_dtype, int kv_dtype, void* out, float* lse, void* workspace,
                     size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Attention of queries over the positions the indexer chose for them.
 *   idx [total_q, k] int32: positions local to the row's request, as the
 *          dsa_index_* calls answer them.  An entry below 0 or beyond the
 *          row's own position is skipped, and one whose page id lies outside
 *          the pool (which is also recorded); one that stands twice counts
 *          twice.
 *   All else as for dsa_attend_paged, without max_q: a request may own any
 *   number of rows (a whole prompt).  1 <= k <= 65536.
 * ---------------------------------------------------------------------- */
int dsa_attend_selected_workspace_size(int B, int total_q, int k, int Hq, int Hkv, int d, int q_dtype, int kv_dtype,
                                       size_t* bytes);
int dsa_attend_selected(const void* Q, const void* K, const void* V, const float* K_scale, const float* V_scale,
                        const int32_t* block_table, const int32_t* lens, const int32_t* q_offsets,
                        const int32_t* idx, int k, int B, int total_q, int n_pages, int page, int64_t page_stride,
                        int max_pages, int Hq, int Hkv, int d, const float* softmax_scale, int q_dtype, int kv_dtype,
                        void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_PAGED_H */
