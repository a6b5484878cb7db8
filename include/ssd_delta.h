/*
 * ssd_delta.h - C ABI of libssd: the gated delta rule, as HIP kernels for MI355X (gfx950).  It stands where the SSD
 * recurrence of ssd.h stands in a stack, on the same states, gates, groups and packed token axis; the conventions of ssd.h
 * for ownership, errors and checks hold here too (ssd_strerror describes the codes).
 *
 * The operator, for every sequence and value head h with key head g = h / (H / G), a_t = exp(log_a[t,h]):
 *
 *     S~_t = a_t S_{t-1}                      S: N x P, fp32
 *     e_t  = v_t - S~_t^T k_t                 what the state does not yet say for the key k_t
 *     S_t  = S~_t + beta_t k_t e_t^T
 *     y_t  = scale S_t^T q_t
 *
 * that is S_t = a_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T.  The state stays bounded for beta_t |k_t|^2 in
 * [0, 2]: keys are of unit length and beta in [0, 1] in common use; the kernels do not normalise and do not check.  What fp32
 * keeps there: errors of states and fp32 gradients are about 1e-6 of their 2-norm with keys apart, at any such beta; with one key for all
 * of a chunk's tokens 3e-6 for beta in [1, 2], and up to 5e-5 where all of them are 2 (its triangular system is ill-conditioned then).
 * The forward and backward passes evaluate it in chunks of 64 tokens on the matrix unit; the result does not depend on that
 * but in rounding.
 *
 * Layouts: q, k [total, G, N], v, y [total, H, P] in `dtype`; log_a, beta [total, H] fp32; states [nseq, H, N, P] fp32.
 * One token's heads are dense, and q, k and v may be views of wider rows with a token stride of their own; everything
 * else is dense.  Values: log_a <= 0 (below -160 it is taken as that, a decay of zero in fp32); an infinity or NaN in an
 * input may reach every output of its own sequence (of its own head; through a key or query, of its group), and none
 * of another.  Precision: states, gates, their gradients and all sums fp32; with bf16 inputs products of computed values
 * take them in three bf16 terms, which hold an fp32's 24 bits, and what only bf16 outputs are made of (y in the forward pass, dq and
 * dk) in two: 2^-16 of each operand, so that those outputs are off by their own rounding.
 * dlog_a is a difference of sums over its chunk: its rounding is relative to those, not to itself.
 * Outputs and the workspace must not overlap inputs or each other; a call where one of them is the very pointer of
 * an input or of another output is refused (SSD_ERR_INVALID), but for final_state, which may be init_state itself.
 * Tokens of no sequence are never written.  No sum is made by atomics: equal calls give equal bits.
 */
#ifndef SSD_DELTA_H
#define SSD_DELTA_H

#include "ssd.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int64_t nseq;      /* sequences, >= 0 */
    int64_t total;     /* tokens of the packed axis, 0 .. 2^31 - 1025 (ssd_delta_step: ignored, one for each sequence) */
    int64_t nheads;    /* H >= 1 */
    int64_t ngroups;   /* G >= 1, divides H: key (and query) heads */
    int64_t keydim;    /* N: 32, 64 or 128 */
    int64_t valuedim;  /* P: a multiple of 32, at most 256 */
    int64_t q_stride;  /* elements from one token of q to the next; 0: dense (G N).  A multiple of 16 bytes, at */
    int64_t k_stride;  /* least the token's own elements, under 2^24.  Likewise k, v (dense: H P).  G N and */
    int64_t v_stride;  /* H P are under 2^24 */
    float scale;       /* of y: finite */
    int32_t dtype;     /* ssd_dtype of q, k, v, y and their gradients */
} ssd_delta_dims;

/*
 * Forward over whole sequences (training, prompts).
 *   cu_seqlens   DEVICE memory, nseq + 1 int64 offsets, non-decreasing: sequence s is tokens cu[s] .. cu[s+1] - 1.
 *                NULL: nseq sequences of total / nseq tokens (total must be a multiple).  The host does not read
 *                it; the kernels clamp it into the axis, so malformed offsets give wrong outputs but no access
 *                outside the tensors or the workspace.
 *   init_state   the states before the first tokens, or NULL for zeros.
 *   final_state  the states after the last tokens (init_state of an empty sequence), or NULL to skip them.
 *   workspace    device scratch of at least ssd_delta_forward_workspace_bytes(dims) bytes, 16-byte aligned, private to
 *                calls that may overlap; its contents are undefined afterwards.
 * Two launches.
 */
size_t ssd_delta_forward_workspace_bytes(const ssd_delta_dims* dims);

int ssd_delta_forward(const ssd_delta_dims* dims, const int64_t* cu_seqlens, const void* q, const void* k,
                      const void* v, const float* log_a, const float* beta, const float* init_state, void* y,
                      float* final_state, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The backward pass: the gradients of <dy, y> + <dfinal, final_state> for ssd_delta_forward, whose inputs these are
 * (it needs none of its results).
 *   dy           [total, H, P] dense;  dfinal [nseq, H, N, P] fp32, or NULL for zeros.
 *   dq, dk       [total, G, N] (summed over the value heads of each group);  dv [total, H, P].
 *   dlog_a, dbeta  [total, H] fp32.
 *   dinit        [nseq, H, N, P] fp32, or NULL to skip it.
 *   workspace    at least ssd_delta_backward_workspace_bytes(dims) bytes; chiefly, for every 64 tokens of a head, a state of
 *                fp32 and one of `dtype` (48 KB at 128 by 64, bf16) and four triangular 64 x 64 operands of all terms (96 KB in bf16, 64 in
 *                fp32): 1.27 GB for 8 x 2048 tokens, 24 heads of 128 by 64, 2.08 GB for 16384 tokens, 32/16 heads of 128 by 128 (the
 *                forward pass 0.48 GB for either), bf16.
 * Four launches.
 */
size_t ssd_delta_backward_workspace_bytes(const ssd_delta_dims* dims);

int ssd_delta_backward(const ssd_delta_dims* dims, const int64_t* cu_seqlens, const void* q, const void* k,
                       const void* v, const float* log_a, const float* beta, const float* init_state, const void* dy,
                       const float* dfinal, void* dq, void* dk, void* dv, float* dlog_a, float* dbeta, float* dinit,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * One token for each sequence (a decode step): state [nseq, H, N, P] is read and overwritten; q, k [nseq, G, N],
 * v, y [nseq, H, P], log_a, beta [nseq, H].  dims->total is ignored.  One launch.
 */
int ssd_delta_step(const ssd_delta_dims* dims, float* state, const void* q, const void* k, const void* v,
                   const float* log_a, const float* beta, void* y, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSD_DELTA_H */
