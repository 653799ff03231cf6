/*
 * tfx_rope — rotary positions of the rows that the q/k/v group gives, ahead of
 * attention and of the cache's appends (tfx_attn.h), for GB300 (sm_103a).
 *
 * Conventions are those of tfx_exl3.h: 0 or a negative TFX_E* code, nothing
 * enqueued after a validation error, tfx_exl3_last_error() for the message;
 * tensor data is caller-owned device memory; calls allocate nothing and can be
 * captured in a CUDA graph.
 */
#ifndef TFX_ROPE_H
#define TFX_ROPE_H

#include "tfx_exl3.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Of each head, the first `rotary` values are rotary/2 pairs, value i with value
 * i + rotary/2, or (interleaved) 2i with 2i + 1. Pair i of a row at position n:
 *     (a, b) -> gain * (a cos w - b sin w, b cos w + a sin w),  w = n * freqs[i].
 * rotary is a multiple of 16 (TFX_EUNSUPPORTED otherwise), at most 2,048.
 * table: rotary/2 values made by tfx_rope_table, in device memory. */
typedef struct {
  const uint64_t* table;
  int rotary, interleaved;
  float gain;
} tfx_rope;

/* The n frequencies (radians a position, finite, host memory) as fractions of a
 * turn in 64 bits (host memory). A position times such a fraction wraps exactly, so an
 * angle has the frequency's own rounding (2^-52 of it, in 64-bit floating point) and
 * FP32's, however far the position. Scalings for long contexts are the caller's choice
 * of frequencies and gain. Host only. */
int tfx_rope_table(const double* freqs, int n, uint64_t* table);

/* Rows of q (heads_q heads of dim values next to each other, ldq elements apart)
 * and of k (heads_k; 0 where there is none) to q_out and k_out: row t is at position
 * positions[t] (device; any int32). Values behind the first `rotary` of a head are
 * copied. An output may be its own input, with the same pitch; else it overlaps no
 * other tensor of the call.
 * dim, pitches: multiples of 8, pointers 16-byte aligned (TFX_EALIGN otherwise);
 * act: tfx_dtype. FP32 inside, rounded once.
 * inverse: rotates by -w instead, with the same gain: the transpose, which the
 * gradient needs, and the inverse where gain is 1. */
int tfx_rope_apply(const tfx_rope* r, int act, int dim, const void* q, int64_t ldq, int heads_q, void* q_out, int64_t ldqo,
                   const void* k, int64_t ldk, int heads_k, void* k_out, int64_t ldko, const int32_t* positions, int rows,
                   int inverse, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* TFX_ROPE_H */
