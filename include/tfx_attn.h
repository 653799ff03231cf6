/*
 * tfx_attn — causal attention over packed prompts, attention of single tokens
 * over a paged K/V cache whose sequences share a prefix, and that cache's page
 * operations, for GB300 (sm_103a). Between the q/k/v group and o_proj of
 * tfx_exl3.h these take the place of the stand-ins: rows of q, k and v are the
 * group's outputs as they are, rows of the attention output are o_proj's input.
 *
 * Conventions are those of tfx_exl3.h: 0 or a negative TFX_E* code, nothing
 * enqueued after a validation error, tfx_exl3_last_error() for the message;
 * pointers to tensor data are caller-owned device memory unless stated
 * otherwise; everything is enqueued on `stream`; calls allocate nothing (only
 * tfx_cache_reserve does) and can be captured in a CUDA graph.
 */
#ifndef TFX_ATTN_H
#define TFX_ATTN_H

#include "tfx_exl3.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Heads of one attention call. Query head h reads K/V head h / (heads_q /
 * heads_kv); heads_kv divides heads_q, at most 128 query heads share one.
 * dim: 128 or 256 (TFX_EUNSUPPORTED otherwise). act: tfx_dtype of every tensor. */
typedef struct {
  int heads_q, heads_kv, dim, act;
  float scale; /* of the scores; finite and positive */
} tfx_attn_heads;

/* Causal attention over n packed sequences: sequence i is the rows
 * offsets[i] .. offsets[i+1]-1, and for its row t and head h
 *     out[t][h] = sum_j p_j v[j][h'],  p = softmax_j(scale * q[t][h] . k[j][h']),
 * over the rows j <= t of the same sequence (h' = h / (heads_q/heads_kv)).
 * offsets : HOST memory, n+1 values, offsets[0] >= 0, not decreasing; equal
 *           neighbours are an empty sequence. Rows outside are not touched.
 * q, out  : rows of heads_q*dim values, ldq / ldo elements apart; k, v: rows of
 *           heads_kv*dim values, ldk / ldv apart. Every pitch a multiple of 8
 *           elements and every pointer 16-byte aligned (TFX_EALIGN otherwise),
 *           so slices of one packed q/k/v buffer are fine. out must not overlap
 *           the inputs.
 * Scores, softmax and sums are FP32; the probabilities are rounded to `act`
 * for the product with v (as matrix operands), the output once. Bits do not
 * depend on the other sequences of the call. */
int tfx_attn_prompt(const tfx_attn_heads* h, const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v,
                    int64_t ldv, const int32_t* offsets, int n, void* out, int64_t ldo, cudaStream_t stream);

/* A paged K/V cache. All memory but priv is the caller's.
 * k, v  : [layers][pages][page_size][heads_kv][dim] in act, 16-byte aligned;
 *         page_size 16, 32, 64 or 128; dim 128 or 256.
 *         pages * page_size and slots * width below 2^31, width * page_size at
 *         most 2^31 - 2048, and that times the batch of a decode call below
 *         2^31 * 4096 / dim (TFX_EUNSUPPORTED otherwise).
 * book  : int32[tfx_cache_book_ints()], device:
 *           [0] status bits, kept until the caller clears them (TFX_CACHE_*);
 *           [1] pages moved by the last compact; [2], [3] unused;
 *           [4 ..] tokens held by each of `slots` sequence slots; then the
 *           reference count of each page; then the page table of each slot,
 *           `width` entries, -1 where it has no page.
 *         An empty cache: all zero, tables -1. Reference counts say in how many
 *         tables a page is; 0 is a free page.
 * priv  : library state, NULL until tfx_cache_reserve().
 * Calls on one cache are ordered on one stream. Slot and page numbers come
 * from device memory and are checked there: one that is out of range, or a
 * sequence that finds no room, is left as it was and leaves a status bit. */
typedef struct {
  void* k;
  void* v;
  int32_t* book;
  int layers, pages, page_size, heads_kv, dim, act;
  int slots, width;
  void* priv;
} tfx_cache;

#define TFX_CACHE_FULL 1       /* no free page was left for a sequence */
#define TFX_CACHE_BAD 2        /* a slot, page or offset out of range, or a fork onto a slot in use */
#define TFX_CACHE_TABLE_FULL 4 /* a sequence would need more than `width` pages */

#define TFX_ATTN_MAX_BATCH 4096

int64_t tfx_cache_book_ints(const tfx_cache* c);

/* Grow-only scratch for tfx_attn_decode over up to max_batch sequences of
 * heads_q query heads, and for the page calls. max_batch <= TFX_ATTN_MAX_BATCH. */
int tfx_cache_reserve(tfx_cache* c, int max_batch, int heads_q, cudaStream_t stream);
int tfx_cache_release(tfx_cache* c);

/* Room for new tokens: sequence seqs[i] (device, distinct slots) grows by
 * offsets[i+1] - offsets[i] tokens (device, n+1 values from 0 up). New pages
 * are the free ones of lowest number, in the order of the list. A sequence
 * that finds too few, or whose table is full, keeps its length. Pages are counted
 * down the list as they are asked for: behind a sequence that finds too few, every
 * one that needs a page finds none either (TFX_CACHE_FULL), however few it needs. A
 * caller puts what must not be refused first. */
int tfx_cache_extend(tfx_cache* c, const int32_t* seqs, const int32_t* offsets, int n, cudaStream_t stream);

/* The new tokens' K and V of one layer, after the extend that made room for
 * them: row t of k and v (heads_kv*dim values, ldk / ldv elements apart, both
 * multiples of 8) is the token that the lists of the last tfx_cache_extend give
 * row t. Rows of sequences that extend left as they were, and rows past its last
 * offset, are not stored. Other calls may come in between (a compact too); a row
 * whose slot has since been freed, forked onto, or extended by another number of
 * tokens is not stored and leaves TFX_CACHE_BAD. A fork copies the tokens of a
 * partly filled page as they are: fork a sequence after its appends. */
int tfx_cache_append(tfx_cache* c, int layer, const void* k, int64_t ldk, const void* v, int64_t ldv, int rows,
                     cudaStream_t stream);

/* The same with lists of its own (device; n as in tfx_cache_extend): where
 * several extends have made room, the lists of the one that these rows are for, or
 * some of its entries. Rows offsets[i] .. offsets[i+1]-1 are the tokens that the last
 * extend of sequence seqs[i] made room for: as many, or none is stored. */
int tfx_cache_append_listed(tfx_cache* c, int layer, const void* k, int64_t ldk, const void* v, int64_t ldv, int rows,
                            const int32_t* seqs, const int32_t* offsets, int n, cudaStream_t stream);

/* dst[i] becomes a copy of sequence src[i] (device lists; dst distinct, empty
 * slots that are in no src): full pages are shared, a last page that is partly
 * filled is copied to the free page of lowest number, in the order of the list. */
int tfx_cache_fork(tfx_cache* c, const int32_t* src, const int32_t* dst, int n, cudaStream_t stream);

/* The sequences give their pages back (device list); a page is free when its
 * last sequence has left. */
int tfx_cache_free(tfx_cache* c, const int32_t* seqs, int n, cudaStream_t stream);

/* Moves used pages to the front of the pool: with L pages in use, the used
 * pages from L on go, in order, to the free pages below L, and every table is
 * brought in line. book[1] is the number of pages moved. */
int tfx_cache_compact(tfx_cache* c, cudaStream_t stream);

/* Contents of page src[i] to page dst[i], all layers, K and V (device lists;
 * dst distinct and none of them in src). Tables and counts stay. */
int tfx_cache_copy(tfx_cache* c, const int32_t* src, const int32_t* dst, int n, cudaStream_t stream);

/* Attention of one new token of each of `batch` sequences over the cache of
 * `layer`: for sequence s = seqs[i] (device), row i of q (heads_q*dim values,
 * ldq elements apart) attends to all tokens s holds, its newest included.
 * shared: the first `shared` tokens are the same in every sequence of the
 * batch (they come from one fork): they are read through the table of the
 * first sequence that holds them all, once for every 256 rows of a K/V head (batch *
 * heads_q/heads_kv) where it has more than 32 and there are 256 such tokens or more,
 * else once for every 16 rows; 0 where nothing is shared. A sequence shorter than
 * that attends to as many of them as its length says (what it does not hold of
 * them must then be finite). A sequence that holds no token, or a slot out of
 * range, gives zeros. h->heads_kv, dim and act are the cache's. Same arithmetic as
 * tfx_attn_prompt, with partial results of FP32 joined in a fixed order. */
int tfx_attn_decode(tfx_cache* c, int layer, const tfx_attn_heads* h, const void* q, int64_t ldq, const int32_t* seqs,
                    int batch, int shared, void* out, int64_t ldo, cudaStream_t stream);

/* The cache's device error word is one for the library: 0, or 1 when an
 * attention kernel gave up a bounded wait (see tfx_exl3_debug_set_spin_limit);
 * its outputs are then not valid. Reading clears it. Synchronous; for tests and
 * diagnostics. */
int tfx_attn_debug_error(int* device_error);

#ifdef __cplusplus
}
#endif
#endif /* TFX_ATTN_H */
