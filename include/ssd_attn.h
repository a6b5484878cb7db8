/*
 * ssd_attn.h - C ABI of libssd: the attention layer of a hybrid stack, as HIP kernels for MI355X
 * (gfx950).  Hybrid stacks put one attention layer after every few SSD layers (llms.blog "State Space
 * Models and Mamba", on hybrid architectures), over the same tokens; these entry points run on the
 * token axes, offsets, element types and streams of ssd.h, whose conventions for ownership, errors and
 * checks hold here too (ssd_strerror describes the codes).
 *
 * The operator, for query i and key j of one sequence (a document of a packed batch), head h with
 * key/value head h / (H / Hk):
 *
 *     z_ij = scale q_i . k_j
 *     s_ij = (softcap > 0 ? softcap tanh(z_ij / softcap) : z_ij) + bias_h(pk_j - pq_i)
 *     p_ij = exp(s_ij - lse_i),   lse_i = log sum_j exp s_ij over the keys visible to i
 *     y_i  = sum_j p_ij v_j
 *
 * Positions: pk_j = j, pq_i = i + Lk - Lq within the sequence: its Lq queries are the last Lq of its Lk
 * positions.  Visible: every key of the same sequence, and with `causal` only those with pk_j <= pq_i,
 * or pk_j < prefix of the sequence when prefixes are given.  A query that sees no key has y = 0,
 * lse = -infinity, and no part in any gradient.
 *
 * Bias, one of: none; slopes [H], bias = -slopes[h] |pk_j - pq_i|; a learned table [num_buckets, H],
 * bias = table[bucket(pk_j - pq_i), h].  Buckets: bidirectional = 0: n = num_buckets, distance
 * d = max(pq_i - pk_j, 0).  bidirectional = 1: n = num_buckets / 2, d = |pk_j - pq_i|, and keys behind the
 * query (pk_j > pq_i) take the table's second half.  With e = n / 2 and f = n - e: d < e has bucket d; d >= e
 * has bucket e + k for the largest k < f with (max_distance / e)^k <= (d / e)^f, that is distances spaced
 * evenly in the logarithm up to max_distance and one bucket beyond; the borders are found in whole
 * numbers, not in rounded logarithms.
 *
 * Layouts: q, y [total_q, H, D], k, v [total_k, Hk, D]; one token's heads are dense, and q, k, v may be
 * views of wider rows (a fused projection's output) with a token stride of their own.  Everything else
 * is dense.  slopes, table and lse are fp32 whatever the dtype.
 * Outputs and the workspace must not overlap inputs or each other; a call where one of them is the very pointer of
 * an input (offsets, lengths and tables among them) or of another output is refused (SSD_ERR_INVALID).
 * Sizes: a launch holds under 2^24 workgroups (2^23 in the backward pass of 128-wide bf16 heads), one for each sequence
 * and each further 128 of its queries or keys, of each head (in forward and decode of each group of heads, where they share
 * keys); calls past that are SSD_ERR_UNSUPPORTED.  Tokens to append are not limited by it.
 * Non-finite inputs: y and lse of a query depend on that query and on the keys and values it sees, whatever
 * the others hold, to the bit.  An infinity in a value that a query of ssd_attn_forward sees is that column of its y
 * (NaN beside one of the other sign or a NaN).  Gradients: an infinity or NaN may reach every gradient of its own sequence
 * and key/value head.  Inputs outside every sequence reach no output.  Sums over the keys are fp32 and divided at the
 * end: 2^8 |v| times the number of keys has to stay under 2^127.
 */
#ifndef SSD_ATTN_H
#define SSD_ATTN_H

#include "ssd.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int64_t nseq;          /* sequences, >= 0 */
    int64_t total_q;       /* tokens of the packed query axis, 0 .. 2^31 - 1025 */
    int64_t total_k;       /* tokens of the packed key axis, 0 .. 2^31 - 1025 */
    int64_t nheads;        /* H >= 1 */
    int64_t nkvheads;      /* Hk >= 1, divides H */
    int64_t headdim;       /* D: 32, 64 or 128 */
    int64_t q_stride;      /* elements from one token of q to the next; 0: dense (H D).  A multiple of */
    int64_t k_stride;      /* 16 bytes, at least the token's own elements, under 2^24.  Likewise k, v */
    int64_t v_stride;      /* (dense: Hk D).  H D itself is under 2^24 */
    float scale;           /* of q . k: finite */
    float softcap;         /* 0: none; else positive and finite (taken as 2^-56 below that, as 2^96 above) */
    int32_t dtype;         /* ssd_dtype of q, k, v, y and their gradients */
    int32_t causal;        /* 0 or 1 */
    int32_t num_buckets;   /* with a table: 2 .. 64 (bidirectional: 4 .. 128, even), otherwise ignored */
    int32_t max_distance;  /* with a table: above half a direction's buckets, at most 1024 */
    int32_t bidirectional; /* with a table: 0 or 1 */
} ssd_attn_dims;

/*
 * Attention forward (for training and prompts).
 *   cu_seqlens_q  DEVICE memory, nseq + 1 int64 offsets into the query axis, non-decreasing; sequence s is
 *                 tokens cu[s] .. cu[s+1] - 1.  NULL: nseq sequences of total_q / nseq tokens (total_q
 *                 must be a multiple).  The host does not read it; the kernels clamp it into the axis, so
 *                 malformed offsets give wrong outputs but no access outside the tensors.
 *   cu_seqlens_k  the same for the key axis.  NULL: cu_seqlens_q (total_k must equal total_q), or equal
 *                 sequences when that is NULL too; given without cu_seqlens_q: SSD_ERR_INVALID.
 *   prefix        DEVICE memory, nseq int64 prefix lengths in keys, or NULL; needs causal = 1.
 *   slopes, table at most one is given.
 *   lse           [total_q, H] output, natural logarithm, or NULL (the backward pass needs it).
 * Tokens of no sequence are never written.  No workspace; one launch.
 */
int ssd_attn_forward(const ssd_attn_dims* dims, const int64_t* cu_seqlens_q,
                     const int64_t* cu_seqlens_k, const int64_t* prefix, const void* q,
                     const void* k, const void* v, const float* slopes, const float* table,
                     void* y, float* lse, void* stream);

/*
 * The backward pass of ssd_attn_forward: the gradients of <dy, y> with respect to q, k, v and the table
 * (of the learned bias; slopes and scale are constants), for training.
 *   q .. table    the forward pass's inputs;  y, lse  its outputs;  dy [total_q, H, D] dense.
 *   dq            [total_q, H, D];  dk, dv [total_k, Hk, D] (summed over the heads of each group).
 *   dtable        [num_buckets, H] fp32, or NULL to skip it; needs table.
 *   workspace     device scratch of at least ssd_attn_backward_workspace_bytes(dims, dtable wanted)
 *                 bytes, 16-byte aligned; its contents are undefined afterwards.
 * Rows of no sequence are never written; a key that no query sees has zero gradients.  No sum is made
 * by atomics: equal calls give equal bits.  Two to five launches.
 */
size_t ssd_attn_backward_workspace_bytes(const ssd_attn_dims* dims, int want_dtable);

int ssd_attn_backward(const ssd_attn_dims* dims, const int64_t* cu_seqlens_q,
                      const int64_t* cu_seqlens_k, const int64_t* prefix, const void* q,
                      const void* k, const void* v, const float* slopes, const float* table,
                      const void* y, const float* lse, const void* dy, void* dq, void* dk, void* dv,
                      float* dtable, void* workspace, size_t workspace_bytes, void* stream);

/*
 * A paged cache of keys and values: k_cache, v_cache [num_pages, page_size, Hk, D].  Position t of sequence s
 * is row t % page_size of page block_table[s, t / page_size] (block_table: DEVICE memory, int32
 * [nseq, max_pages]).  An entry that is no page (negative, or num_pages and more) is never followed: its
 * keys are not visible, and nothing is written to it.
 */
typedef struct {
    int64_t nseq;          /* sequences, >= 0 */
    int64_t nheads;        /* H, Hk, D as in ssd_attn_dims */
    int64_t nkvheads;
    int64_t headdim;
    int64_t num_pages;     /* 0 .. 2^31 - 1 */
    int64_t page_size;     /* a multiple of 16, at most 65536 */
    int64_t max_pages;     /* entries of a block table row, >= 0; max_pages page_size at most 2^31 - 1025 */
    int64_t q_stride;      /* elements from one token to the next, as in ssd_attn_dims (0: dense) */
    int64_t k_stride;      /* of the tokens that ssd_kv_append is given */
    int64_t v_stride;
    float scale;
    float softcap;
    int32_t dtype;         /* ssd_dtype of q, k, v, y and the cache */
    int32_t num_buckets;   /* with a table: as in ssd_attn_dims */
    int32_t max_distance;
    int32_t bidirectional;
} ssd_attn_cache;

/*
 * Attention of one query per sequence over the cache (a decode step): the operator above with Lq = 1 and
 * Lk = seq_lens[s], every cached position visible, the query at the last one.
 *   q [nseq, H, D], y [nseq, H, D] dense; block_table, seq_lens (int64 [nseq], clamped into
 *   [0, max_pages page_size]) DEVICE memory, read by the kernels only.  A sequence of no visible key has y = 0.
 *   Rows of a page past a sequence's length are not read.
 *   workspace     ssd_attn_decode_workspace_bytes(dims) bytes, 16-byte aligned, private to calls that
 *                 may overlap; its contents are undefined afterwards.
 * One launch, or two where sequences are split along their keys.
 */
size_t ssd_attn_decode_workspace_bytes(const ssd_attn_cache* dims);

int ssd_attn_decode(const ssd_attn_cache* dims, const void* q, const void* k_cache,
                    const void* v_cache, const int32_t* block_table, const int64_t* seq_lens,
                    const float* slopes, const float* table, void* y, void* workspace,
                    size_t workspace_bytes, void* stream);

/*
 * Appends new tokens' keys and values to the cache, the keys rotated by their positions, and rotates the
 * queries beside them.  Tokens are packed: token i of sequence s (cu_seqlens, int64 [nseq + 1], DEVICE
 * memory; NULL: one token per sequence, tokens must equal nseq) has position
 * seq_lens[s] - (cu_seqlens[s + 1] - i): seq_lens counts the sequence with its new tokens.
 *   inv_freq      fp32 [rot_pairs] or NULL (no rotation, rot_pairs 0): pair r of a head is turned by
 *                 position * inv_freq[r] radians, (a, b) -> (a cos - b sin, b cos + a sin).
 *   rot_pairs     a multiple of 8, at most D / 2.  Pairs are elements (r, r + rot_pairs), or with
 *                 `interleaved` (2 r, 2 r + 1); elements from 2 rot_pairs on are copied.
 *   q, q_out      queries [tokens, H, D] and their rotated copy (dense), or both NULL.
 * A token whose position is outside the block table or on no page is not appended (its query is rotated
 * all the same); tokens of no sequence are left alone.  Two tokens for one place leave either's values,
 * element by element.
 */
int ssd_kv_append(const ssd_attn_cache* dims, int64_t tokens, const int64_t* cu_seqlens,
                  const int64_t* seq_lens, const int32_t* block_table, const void* k, const void* v,
                  const void* q, const float* inv_freq, int rot_pairs, int interleaved,
                  void* k_cache, void* v_cache, void* q_out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSD_ATTN_H */
