/*
 * ssd_rotary.h - C ABI of libssd: rotary positions of queries and keys, for training and prompts, on MI355X (gfx950).
 * ssd_kv_append rotates as it writes a cache; this is the rotation by itself, beside ssd_attn_forward and its backward pass.
 *
 * For pair r of a head's rot_pairs, at position p of its sequence:
 *
 *     (a, b) -> m (a cos t - b sin t, b cos t + a sin t),   t = p inv_freq[r]
 *
 * with m the magnitude of a context scaled beyond the one trained on (1 without; the appends to a cache have none: where all of a
 * head is rotated take m^2 into the attention's scale, else rotate here and append without frequencies).  Pairs are elements (r, r + rot_pairs), or with
 * `interleaved` (2 r, 2 r + 1); elements from 2 rot_pairs on are copied.  With `inverse` the angle is -t: the gradient of
 * the rotation, taken of the gradients of its outputs.  Angles are reduced in fp64, so that far positions keep theirs.
 */
#ifndef SSD_ROTARY_H
#define SSD_ROTARY_H

#include "ssd.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int64_t nseq;        /* sequences, >= 0 */
    int64_t total;       /* tokens of the packed axis, 0 .. 2^31 - 1025 */
    int64_t nheads;      /* H >= 1, of q */
    int64_t nkvheads;    /* Hk >= 1, of k (ignored without k) */
    int64_t headdim;     /* D: 32, 64 or 128 */
    int64_t q_stride;    /* elements from one token to the next; 0: dense.  A multiple of 16 bytes, at least the token's */
    int64_t k_stride;    /* own elements, under 2^24 */
    float magnitude;     /* m: finite */
    int32_t dtype;       /* ssd_dtype */
    int32_t rot_pairs;   /* a multiple of 8, 0 .. D / 2 */
    int32_t interleaved; /* 0 or 1 */
    int32_t inverse;     /* 0 or 1 */
} ssd_rotary_dims;

/*
 *   cu_seqlens  DEVICE memory, nseq + 1 int64 offsets, or NULL: nseq sequences of total / nseq tokens (total must be a
 *               multiple).  Read by the kernels only; tokens of no sequence are not written.
 *   start       DEVICE memory, nseq int64 positions of the sequences' first tokens (what came before, in a cache), or
 *               NULL for zeros.
 *   q, q_out    [total, H, D], q_out dense;  k, k_out  [total, Hk, D], or both NULL.
 *   inv_freq    fp32 [rot_pairs], or NULL with rot_pairs 0.
 * Outputs must not overlap inputs or each other (SSD_ERR_INVALID where one is the very pointer of another).  One launch.
 */
int ssd_rotate(const ssd_rotary_dims* dims, const int64_t* cu_seqlens, const int64_t* start, const void* q, const void* k,
               const float* inv_freq, void* q_out, void* k_out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSD_ROTARY_H */
