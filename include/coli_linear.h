/* coli_linear -- y = W x for few tokens with W in 4-bit codes and group scales, on an NVIDIA GB300 (sm_103a), C ABI.
 *
 * The dense products of a decoder layer around its attention and experts (query, key and value projection, output
 * projection, logits) when it answers token by token:
 *
 *   y[t,n] = sum over groups g of s[n,g] * sum over k in g of c[n,k] * x[t,k]
 *
 * Format.  c are codes in -8..7, two's-complement nibbles, column 2i in the low nibble of byte i of its row (as the
 * experts' int4 rows); s is one scale of the activations' type for each row and group of 32, 64 or 128 consecutive columns.
 * The library keeps its own copy of both in its device layout.
 *
 * Numbers.  x, s and y are bf16 or fp16 (one type per handle).  Codes and x multiply exactly; sums are fp32, over a group
 * first, which its scale then multiplies; y is rounded once.  The order of the sums depends on the shape and on whether a call
 * has up to 8, up to 16 or more tokens, not on the other tokens, and equal calls give equal bits.
 *
 * A call of up to 16 tokens (8, with more than 24576 columns) reads the weights once; a larger one reads them once for every 64
 * tokens with groups of 128, else for every 16 (8), from L2 as far as they fit.
 *
 * Conventions are those of coli_moe.h.  forward allocates nothing, keeps nothing between calls and may be captured in a CUDA
 * graph; calls on one handle may overlap in time, but not with coli_linear_load.
 */
#ifndef COLI_LINEAR_H
#define COLI_LINEAR_H

#include <stdint.h>

#include "coli_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct coli_linear coli_linear; /* the weights in the library's layout; owned by the library */

typedef struct {
  int rows;       /* outputs n, 1..16777216                                  */
  int cols;       /* inputs k, a multiple of group, at most 32768            */
  int group;      /* 32, 64 or 128                                           */
  int dtype;      /* COLI_ATTN_BF16 or COLI_ATTN_FP16                        */
  int max_tokens; /* largest n_tokens of a call, 1..1000000                  */
} coli_linear_config;

/* Validates cfg and allocates the store on the current device (the codes and scales, rows padded to 8 and columns to 128).
 * EINVAL: a value out of the ranges above.  EUNSUPPORTED: group, dtype or cols that the kernels do not cover.  ENOMEM, ECUDA.
 * On error *out is left NULL. */
int coli_linear_create(const coli_linear_config* cfg, coli_linear** out);

/* Frees the handle (synchronises the device first).  NULL is a no-op. */
void coli_linear_destroy(coli_linear* h);

/* Loads the weights: packed_dev [rows, cols/2] bytes and scales_dev [rows, cols/group] of the handle's type, contiguous; packed_dev
 * 4-byte aligned.  Returns when the copy is complete on `stream` (it synchronises it); the caller's memory may then be freed. */
int coli_linear_load(coli_linear* h, const uint8_t* packed_dev, const void* scales_dev, void* stream);

/* y_dev [n_tokens, rows] = W x_dev [n_tokens, cols].  *_stride: elements between tokens; x_stride a multiple of 8 and x_dev 16-byte
 * aligned.  n_tokens == 0 is a no-op.  x and y must not overlap (their rows may lie between one another).  ESTATE: no
 * weights loaded yet. */
int coli_linear_forward(const coli_linear* h, const void* x_dev, int64_t x_stride, int n_tokens, void* y_dev,
                        int64_t y_stride, void* stream);

/* COLI_OK, or COLI_ETIMEOUT if a bounded wait of an earlier call gave up (that call's output is undefined; the word is then cleared).
 * Synchronises `stream`. */
int coli_linear_status(coli_linear* h, void* stream);

/* Packs fp32 rows into the format: s = max|w| / 7 over a group, rounded to dtype, c = round(w / s) (half away from zero) clamped to
 * [-7, 7].  w_dev [rows, cols] -> packed_dev [rows, cols/2], scales_dev [rows, cols/group]; a group of zeros has s = 0.
 * w_dev finite and within dtype's range. */
int coli_linear_quantize(const float* w_dev, int64_t rows, int cols, int group, int dtype, uint8_t* packed_dev,
                         void* scales_dev, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* COLI_LINEAR_H */
