/*
 * kda_attn.h -- C ABI of libkda's softmax attention on AMD Instinct MI355X
 * (gfx950), for the layers that stand between recurrent ones: causal attention
 * over prompts, attention of one or several drafted tokens per request over a
 * paged cache of keys and values, the store of new keys and values into that
 * cache, and its block tables and slots, built on the device from the requests'
 * lengths.
 *
 * They share the rules of kda.h and kda_ssm.h: plain pointers and sizes; every
 * buffer is the caller's device memory; the library allocates nothing and keeps
 * no pointer or state between calls; work is enqueued on `stream` with no host
 * synchronisation, so a call can be captured in a HIP graph without warm-up;
 * argument errors are found on the host before anything is enqueued (the
 * *_validate functions make the same checks and touch no device; pointers are
 * compared, never dereferenced); base pointers are 16-byte aligned; buffers a
 * call writes overlap no other buffer.  A buffer with a row stride counts as its
 * whole span, first element to last.  KDA_ERR_TOO_LARGE: 2^31 tokens, pages or
 * table rows or more, more than 2^30 positions in a table's row, packed rows of 2^23 elements or
 * more, or so much work that a launch would have 2^32 threads.
 *
 * Batches of prompts are fixed or packed, and offsets are treated, as kda_ssm.h
 * says under Sequences.
 *
 * Heads.  H query heads share num_kv_heads heads of keys and values, H / num_kv_heads
 * neighbours each.  head_dim is 64 or 128.
 *
 * Accuracy.  Scores, the softmax's maxima and sums and the outputs' sums are
 * fp32.  A weight exp(s - m) is rounded to bf16 ahead of the product with the
 * values (the sum that divides them is of the unrounded ones), an output once.
 * Range.  Products q . k and scores have to be below 2^127 in magnitude.  Values may be of any size up to
 * 2^127 (of rows that see more than 2^22 positions, 2^149 over their number): no sum leaves
 * fp32.  At its other end, with values in bf16, weights below 2^-95 of a row's largest count as
 * zero, and what an output loses is 2^-95 times the positions at most.
 * A score of minus infinity is a weight of zero.  A row of which no other score is left has an lse of minus
 * infinity, and outputs that are NaN (over a cache zeros, as where it sees nothing).  A row that has a score of
 * plus infinity or NaN is NaN, one that sees an infinity or a NaN among the values is infinite or NaN in
 * that column; rows that do not see it are as if it were not there, but for their last bits.
 */
#ifndef KDA_ATTN_H_
#define KDA_ATTN_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * Causal attention over prompts.  Within each sequence, for token t and head h
 * with g = h / (H / num_kv_heads):
 *   s_j = scale q[t, h] . k[j, g] for the sequence's tokens j <= t
 *   out[t, h] = sum_j exp(s_j) v[j, g] / sum_j exp(s_j),  lse[t, h] = log sum_j exp(s_j)
 *
 *   q, out          bf16 [T_total, H, head_dim] with row strides
 *   k, v            bf16 [T_total, num_kv_heads, head_dim] with row strides
 *   cu_seqlens      int32 or int64 [N + 1] or NULL (N equally long sequences)
 *   lse             fp32 [T_total, H] or NULL
 * q, k and v may be columns of one row.  Rows behind the last sequence are
 * neither read nor written. */
typedef struct {
  int32_t num_seqs;          /* N >= 1 */
  int64_t total_tokens;      /* T_total >= 0 */
  int32_t num_heads;         /* H >= 1 */
  int32_t num_kv_heads;      /* >= 1, divides H */
  int32_t head_dim;          /* 64 or 128 */
  float scale;               /* > 0 and at most 2^127 */
  int32_t cu_seqlens_int64;  /* 0: int32 offsets, 1: int64 */
  int64_t q_stride;          /* elements between rows, a multiple of 8, at least the row and below
                                2^23; 0 = the row */
  int64_t k_stride;
  int64_t v_stride;
  int64_t out_stride;
} kda_attn_problem;

kda_status kda_attn_validate(const kda_attn_problem* p, const void* q, const void* k, const void* v,
                             const void* cu_seqlens, const void* out, const float* lse);
kda_status kda_attn_prefill(const kda_attn_problem* p, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                            const void* cu_seqlens, uint16_t* out, float* lse, void* stream);

/* ---------------------------------------------------------------------------
 * The cache.  Keys and values lie in pages of page_size tokens, in two buffers
 * [num_pages, page_size, num_kv_heads, head_dim] of the same strides (they may be halves of one): elements are
 * bf16, or e4m3 codes that stand for code * scale with an fp32 scale > 0 per
 * head.  A token's slot is page * page_size + its place in the page.  A block
 * table int32 [table_rows, table_width] names each request's pages in order: position
 * x of the request in row r is in page table[r, x / page_size].  An entry outside
 * [0, num_pages), and a position past the table's width, name no page. */
typedef enum { KDA_CACHE_BF16 = 0, KDA_CACHE_E4M3 = 1 } kda_cache_dtype;

typedef struct {
  int32_t num_kv_heads;      /* >= 1 */
  int32_t head_dim;          /* 64 or 128 */
  int32_t dtype;             /* kda_cache_dtype */
  int32_t page_size;         /* a power of two in 16..1024 */
  int64_t num_pages;         /* 1 .. 2^31 - 1 */
  int64_t page_stride;       /* elements between pages: a multiple of 16, at least the page and
                                at most 2^40; 0 = page_size token strides */
  int64_t token_stride;      /* elements between a page's tokens: a multiple of 16, at least
                                num_kv_heads * head_dim and below 2^23; 0 = packed */
} kda_kv_cache;

/* Attention of T tokens of each of N requests over the cache, which holds their
 * own keys and values already: request n's tokens are at the positions lens[n]
 * .. lens[n] + T - 1 of its block table's row.  Token i of the request sees
 *   positions below lens[n], and
 *   of its own tokens, those j < T whose bit j is set in tree[n, i] (no tree: j <= i).
 * Positions without a page do not count.  A token that sees nothing has zero
 * outputs and an lse of minus infinity.  rows names the requests' rows in the
 * table (NULL: request n has row n); a request whose row is outside [0, table_rows) is an
 * empty slot of the batch: zero outputs, nothing read.  Lengths below zero count as
 * zero.  T = 1 is a decode step; a chain of drafts needs no tree; a tree of drafts
 * gives each its ancestors' bits and its own.
 *
 *   q, out          bf16 [N * T, H, head_dim] with row strides; out may be exactly q with q's
 *                   stride
 *   table           int32 [table_rows, table_width]
 *   rows            int32 [N] or NULL
 *   lens            int32 [N]
 *   tree            uint64 [N, T], or [T] for all requests, or NULL
 *   k_scale, v_scale  fp32 [num_kv_heads] for an e4m3 cache, else NULL
 *   lse             fp32 [N * T, H] or NULL
 *   workspace       kda_attn_decode_workspace_size bytes: scratch that carries
 *                   nothing between calls and must not be used by two calls in
 *                   flight at once
 * Contexts over tables with room for more than 1024 positions are laid end to end and
 * cut into stretches of the same length, which run side by side; a second launch joins what
 * a cut has parted.  The workspace's size follows from the problem's sizes alone; where the cuts
 * are follows from the lengths too, so that a request's last bits can depend on the other requests'
 * lengths (not on anything else: a call repeated gives the same bits). */
typedef struct {
  int32_t num_seqs;          /* N >= 0 requests */
  int32_t tokens_per_seq;    /* T, 1..64; row n * T + t is token t of request n */
  int32_t num_heads;         /* H >= 1, a multiple of cache.num_kv_heads */
  float scale;               /* as for the prefill; times k_scale likewise, and at least 2^-126 */
  int64_t table_rows;        /* 0 .. 2^31 - 1 */
  int32_t table_width;       /* >= 1; table_width * page_size is at most 2^30 */
  int32_t tree_per_seq;      /* 1: tree is [N, T], 0: [T] */
  int64_t q_stride;          /* as for the prefill */
  int64_t out_stride;
  kda_kv_cache cache;
} kda_attn_decode_problem;

kda_status kda_attn_decode_workspace_size(const kda_attn_decode_problem* p, size_t* bytes);
kda_status kda_attn_decode_validate(const kda_attn_decode_problem* p, const void* q, const void* k_cache,
                                    const void* v_cache, const int32_t* table, const int32_t* rows,
                                    const int32_t* lens, const uint64_t* tree, const float* k_scale,
                                    const float* v_scale, const void* out, const float* lse,
                                    const void* workspace, size_t workspace_bytes);
kda_status kda_attn_decode(const kda_attn_decode_problem* p, const uint16_t* q, const void* k_cache,
                           const void* v_cache, const int32_t* table, const int32_t* rows, const int32_t* lens,
                           const uint64_t* tree, const float* k_scale, const float* v_scale, uint16_t* out,
                           float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Keys and values of T tokens into the cache: token t to slot slots[t]; a slot
 * outside [0, num_pages * page_size) stores nothing.  Slots must be distinct (not checked
 * on the device).  bf16 elements are copied; e4m3 codes are x / scale (in fp32), at most 448 in
 * magnitude, rounded to nearest even (an infinity is stored as 448, a NaN as a NaN).
 *
 *   k, v            bf16 [T, num_kv_heads, head_dim] with row strides
 *   slots           int64 [T]
 *   k_scale, v_scale  fp32 [num_kv_heads] for an e4m3 cache, else NULL */
typedef struct {
  int64_t tokens;            /* T >= 0 */
  int64_t k_stride;          /* elements between rows, a multiple of 8, at least the row and below
                                2^23; 0 = the row */
  int64_t v_stride;
  kda_kv_cache cache;
} kda_kv_store_problem;

kda_status kda_kv_store_validate(const kda_kv_store_problem* p, const void* k, const void* v,
                                 const int64_t* slots, const float* k_scale, const float* v_scale,
                                 const void* k_cache, const void* v_cache);
kda_status kda_kv_store(const kda_kv_store_problem* p, const uint16_t* k, const uint16_t* v,
                        const int64_t* slots, const float* k_scale, const float* v_scale, void* k_cache,
                        void* v_cache, void* stream);

/* ---------------------------------------------------------------------------
 * Pages and slots of new tokens.  Request n has lens[n] tokens in its pages and
 * gets the tokens cu_seqlens[n] .. cu_seqlens[n + 1] - 1 of the batch (NULL: T_total / N tokens
 * each) behind them.  Pages that they open, a request's at multiples of page_size, are taken
 * from the list of free pages in the order of the requests and of their
 * positions, from element free_head on:
 *   table[row, x / page_size] = free_pages[...]   for each position x that opens a page
 *   slots[t] = page * page_size + x % page_size   for each new token t at position x
 *   lens_out[n] = lens[n] + the request's new tokens
 *   head_out = free_head + the pages that were needed
 * Where the list is too short, head_out says by how much (it is past num_free),
 * the pages that are missing are -1 in the table, and their tokens' slots are -1.
 * Positions past the table's width take no page and have the slot -1.  A request
 * whose row is outside [0, table_rows) is an empty slot of the batch: its tokens' slots are
 * -1, its length is kept, nothing else happens.  Slots of rows behind the last
 * sequence are -1.  Lengths below zero count as zero; a table entry below zero names no page.  Rows must be
 * distinct (not checked on the device).
 * Tokens can be given back by a smaller length (drafts that were not taken): positions from it on
 * are assigned anew, and a page that only they had opened is the caller's to free.
 *
 *   lens, lens_out  int32 [N]
 *   rows            int32 [N] or NULL (request n has row n)
 *   cu_seqlens      int32 or int64 [N + 1] or NULL
 *   table           int32 [table_rows, table_width], updated in place
 *   free_pages      int32 [num_free]
 *   free_head, head_out  int32 [1]
 *   slots           int64 [T_total] */
typedef struct {
  int32_t num_seqs;          /* N >= 1 */
  int64_t total_tokens;      /* T_total >= 0 */
  int32_t page_size;         /* a power of two in 16..1024 */
  int32_t table_width;       /* >= 1; table_width * page_size is at most 2^30 */
  int64_t table_rows;        /* 0 .. 2^31 - 1 */
  int64_t num_free;          /* 0 .. 2^31 - 1 */
  int32_t cu_seqlens_int64;  /* 0: int32 offsets, 1: int64 */
} kda_kv_assign_problem;

kda_status kda_kv_assign_validate(const kda_kv_assign_problem* p, const int32_t* lens, const int32_t* rows,
                                  const void* cu_seqlens, const int32_t* table, const int32_t* free_pages,
                                  const int32_t* free_head, const int64_t* slots, const int32_t* lens_out,
                                  const int32_t* head_out);
kda_status kda_kv_assign(const kda_kv_assign_problem* p, const int32_t* lens, const int32_t* rows,
                         const void* cu_seqlens, int32_t* table, const int32_t* free_pages,
                         const int32_t* free_head, int64_t* slots, int32_t* lens_out, int32_t* head_out,
                         void* stream);

#ifdef __cplusplus
}
#endif
#endif /* KDA_ATTN_H_ */
