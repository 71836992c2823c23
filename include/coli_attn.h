/* coli_attn -- attention over a paged key/value cache on an NVIDIA GB300 (sm_103a), C ABI.
 *
 * The other half of the decoder layer whose experts coli_moe.h computes: a layer's new keys and
 * values are appended to a cache kept in pages, and its queries attend to that cache.
 *
 *   append  x' = rotation of x by the token's position (queries and keys), k' and v -> cache
 *   window  o = softmax(scale * q K^T) V over the keys j <= p with p - j < window or j < sinks
 *   prefix  the same over one prefix that all sequences share, then each sequence's own keys;
 *           the shared keys are read and multiplied once for the whole batch
 *
 * A batch is ragged.  Sequence b has the query tokens q_start[b] .. q_start[b+1]-1 (its new
 * tokens, the last ones of its cache) and kv_len[b] cached tokens, the new ones included, so its
 * new token i has position p = kv_len[b] - n_b + i.  Its token j sits in slot j % page of page
 * table[b * table_stride + j / page] of the cache.  These three arrays are read on the device, so
 * a captured graph follows them from replay to replay.
 *
 * Rows.  A query that sees no key (an empty sequence, more new tokens than cached ones, window 0
 * without sinks) gets zeros, and -infinity as its log-sum-exp.  What is in cache slots that a query
 * does not see -- unused slots, later tokens, tokens outside the window -- has no influence on its
 * row, not even infinities and NaN.
 *
 * Numbers.  Inputs, cache and output are bf16 or fp16 (one type per handle).  Products accumulate
 * in fp32; softmax maxima, sums and the output accumulators are fp32; the weights are rounded
 * to the type before they multiply V (the tensor cores' operand type), the output once at the end.
 * Work is split over the keys in a fixed order, so equal calls give equal bits.
 *
 * Conventions are those of coli_moe.h: every call returns COLI_OK or a negative status; device
 * pointers are named *_dev or listed as such; calls are asynchronous on `stream` and allocate
 * nothing (safe to capture in a CUDA graph); calls on one handle must not overlap in time (they
 * share its workspace); the current device must be the one the handle was created on.
 */
#ifndef COLI_ATTN_H
#define COLI_ATTN_H

#include <stdint.h>

#include "coli_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define COLI_ATTN_BF16 0
#define COLI_ATTN_FP16 1

typedef struct coli_attn coli_attn;       /* shapes, rotation and workspace; owned by the library */
typedef struct coli_attn_kv coli_attn_kv; /* a bound cache; owned by the library, its memory is not */

typedef struct {
  int n_q;        /* query heads, a multiple of n_kv, at most 64 * n_kv                           */
  int n_kv;       /* key/value heads, 1..256; query head i reads key head i / (n_q / n_kv)          */
  int head_dim;   /* 64 or 128                                                                    */
  int page;       /* tokens per cache page: 16, 32, 64, 128 or 256                                 */
  int dtype;      /* COLI_ATTN_BF16 or COLI_ATTN_FP16                                              */
  int max_tokens; /* largest n_tokens of a call, 1..4194304                                       */
  int max_seqs;   /* largest n_seqs of a call, 1..4096                                            */
  int rot_dim;    /* leading values of a head that are rotated: 0 or a multiple of 16 <= head_dim   */
  int rot_interleaved; /* 1: pairs (2i, 2i+1); 0: pairs (i, i + rot_dim/2)                          */
  double rope_base;    /* pair i turns by p * rope_base^(-2i/rot_dim); > 0, used without inv_freq   */
  const double* inv_freq; /* host [rot_dim/2] radians per position instead, or NULL; read by create */
} coli_attn_config;

/* The caller's cache memory on the device.  Strides are in elements and multiples of 8; the values
 * of a head's token are contiguous; bases are 16-byte aligned.  So pages may hold their heads one
 * after another or interleaved by token, and K and V may share pages. */
typedef struct {
  void* k;
  void* v;
  int64_t n_pages; /* 1..2^31-2 */
  int64_t k_page_stride, k_head_stride, k_slot_stride;
  int64_t v_page_stride, v_head_stride, v_slot_stride;
} coli_attn_cache;

typedef struct {
  const int32_t* q_start; /* device [n_seqs+1], ascending from 0 to n_tokens                        */
  const int32_t* kv_len;  /* device [n_seqs], 0..max_pages*page                                     */
  const int32_t* table;   /* device [n_seqs][table_stride]: page ids, 0..n_pages-1 where used        */
  int64_t table_stride;   /* >= max_pages, or 0: all sequences share one row                         */
  int32_t n_seqs, max_pages, n_tokens;
  int32_t max_q; /* at least the new tokens of any sequence (picks the kernels and sizes the last one) */
} coli_attn_batch;

/* Validates cfg and allocates the workspace on the current device.  EINVAL: a value out of the
 * ranges above.  EUNSUPPORTED: head_dim, page, dtype, rot_dim or n_q / n_kv > 64 that the kernels
 * do not cover.  ENOMEM, ECUDA.  On error *out is left NULL. */
int coli_attn_create(const coli_attn_config* cfg, coli_attn** out);

/* Frees the handle (synchronises the device first).  NULL is a no-op. */
void coli_attn_destroy(coli_attn* h);

/* Describes the caller's cache memory for the calls below (nothing is copied; the memory stays the
 * caller's and must outlive the binding).  EINVAL: NULL, misaligned or non-positive sizes, strides
 * that let tokens of K, or of V, overlap: in order of size, a stride is at least what the smaller ones
 * span (a dimension of one entry has none, but is given as at least head_dim).  The handle's shapes give the dims. */
int coli_attn_cache_bind(coli_attn* h, const coli_attn_cache* cache, coli_attn_kv** out);
void coli_attn_cache_release(coli_attn_kv* kv);

/* Rotates q_dev [n_tokens, n_q, head_dim] into q_out_dev (which may be q_dev itself; both NULL: no
 * queries) and writes the rotated k_dev [n_tokens, n_kv, head_dim] and v_dev into the cache slots
 * of the batch's new tokens.  *_stride: elements between tokens, multiples of 8; bases 16-byte
 * aligned.  pos_base_dev[0] is added to every position for the rotation alone (the length of a shared
 * prefix that the sequences' own caches follow), or NULL.  Positions below 0 (more new tokens than
 * kv_len) are rotated as such and not stored.  The angle is reduced in 64-bit fixed point: its error
 * does not grow with the position. */
int coli_attn_append(coli_attn* h, const coli_attn_kv* kv, const coli_attn_batch* batch,
                     const void* q_dev, int64_t q_stride, const void* k_dev, int64_t k_stride,
                     const void* v_dev, int64_t v_stride, void* q_out_dev, int64_t q_out_stride,
                     const int32_t* pos_base_dev, void* stream);

/* out_dev [n_tokens, n_q, head_dim] = attention of the batch's queries over its cache: query p sees
 * key j when j <= p and (p - j < window or j < sinks).  window < 0: all keys up to p; window = 0:
 * the sinks alone.  sinks >= 0; scale > 0, and finite times log2(e).  lse_dev [n_tokens, n_q]: natural log-sum-exp of the scaled scores, or
 * NULL.  Strides as in append.  q_dev must not overlap out_dev (their rows may lie
 * between one another).  EUNSUPPORTED: the batch could have 2^31 key tiles (n_kv times its blocks,
 * one or more a sequence, times max_pages * page / 64, or the window's share of that): split the call. */
int coli_attn_window(coli_attn* h, const coli_attn_kv* kv, const coli_attn_batch* batch,
                     const void* q_dev, int64_t q_stride, int window, int sinks, float scale,
                     void* out_dev, int64_t out_stride, float* lse_dev, void* stream);

/* Attention of a batch behind a shared prefix: every query sees all prefix_len_dev[0] tokens of the
 * pages prefix_table_dev [prefix_pages] and the keys up to its own position of its own cache (whose
 * positions count from the end of the prefix; kv_len may be 0).  prefix_len is at most prefix_pages * page.
 * n_tokens <= 8 * max_seqs.  EUNSUPPORTED as for window, prefix_pages included. */
int coli_attn_prefix(coli_attn* h, const coli_attn_kv* kv, const coli_attn_batch* batch,
                     const int32_t* prefix_table_dev, int prefix_pages,
                     const int32_t* prefix_len_dev, const void* q_dev, int64_t q_stride, float scale,
                     void* out_dev, int64_t out_stride, float* lse_dev, void* stream);

/* Device status of the handle: COLI_OK; COLI_EINVAL when an earlier call met lengths, offsets or
 * page ids out of range (lengths are clamped, such a page reads as zeros and is not written; rows of tokens that no
 * sequence has, as when the offsets end before n_tokens, are not written or not complete), or a window or
 * prefix call a sequence of more than max_q new tokens (rows of its output may be missing), or offsets that overlap so often
 * that the call's list of key tiles is full (its output is undefined);
 * COLI_ETIMEOUT when a bounded wait gave up (that call's output is undefined).  The word is then
 * cleared.  Synchronises `stream`. */
int coli_attn_status(coli_attn* h, void* stream);

/* Kernels that coli_attn_append (op 0), coli_attn_window (op 1) or coli_attn_prefix (op 2) launches at most for batches of
 * n_seqs sequences.  EINVAL: bad arguments. */
int coli_attn_launches(const coli_attn* h, int op, int n_seqs);

#ifdef __cplusplus
}
#endif
#endif /* COLI_ATTN_H */
