/*
 * ssd_kv8.h - C ABI of libssd: a paged cache of keys and values held in 8 bits, for MI355X (gfx950): the append that
 * quantises, the decode step that reads it, and the read-back.  The cache of ssd_attn.h in half its bytes (bf16; a quarter in fp32); its
 * conventions for pages, lengths, offsets, streams, errors and checks hold here too.
 *
 * Held, for each token and key head, of its key and its value x [D]:
 *
 *     scale = max |x| (1 / L)      fp32, as 1 / L is; L = 127 (SSD_KV8_INT8) or 448 (SSD_KV8_E4M3); rounded up where it is subnormal
 *     x8    = x / scale            rounded to the nearest value of the type, ties to even; zeros where all are
 *
 * so that it stands for scale x8, off by at most scale / 2 (int8), or 2^-4 of the value and scale 2^-10 (e4m3).  A head with an
 * infinity or NaN has a NaN for its scale and reads as NaN.
 *
 * Layouts: k_cache, v_cache [num_pages, page_size, Hk, D] of one byte, k_scale, v_scale [num_pages, page_size, Hk]
 * fp32.  The dims are ssd_attn_cache's; its dtype is that of q, k, v and y.  D is 32, 64 or 128.
 * Outputs and the workspace must not overlap inputs or each other; a call where one of them is the very pointer of
 * an input or of another output is refused (SSD_ERR_INVALID).
 */
#ifndef SSD_KV8_H
#define SSD_KV8_H

#include "ssd_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SSD_KV8_INT8 = 0,
    SSD_KV8_E4M3 = 1 /* 4 exponent bits, bias 7, 3 mantissa bits, no infinity, largest value 448 */
} ssd_kv8_format;

typedef struct {
    void* k;        /* [num_pages, page_size, Hk, D] */
    void* v;
    float* k_scale; /* [num_pages, page_size, Hk] */
    float* v_scale;
    int32_t format; /* ssd_kv8_format */
} ssd_kv8_pages;

/*
 * ssd_kv_append into 8-bit pages: the keys rotated by their positions (in fp32, not rounded between), keys and values
 * quantised, and the queries rotated beside them.  Arguments as there.
 */
int ssd_kv8_append(const ssd_attn_cache* dims, const ssd_kv8_pages* pages, int64_t tokens, const int64_t* cu_seqlens,
                   const int64_t* seq_lens, const int32_t* block_table, const void* k, const void* v, const void* q,
                   const float* inv_freq, int rot_pairs, int interleaved, void* q_out, void* stream);

/*
 * ssd_attn_decode over 8-bit pages: the operator of ssd_attn.h on the values that the pages stand for.  Arguments as
 * there; the workspace from its own query.  Scores, softmax and sums are fp32; the weights of a bf16 call hold 16 bits or more in its
 * products (2^-16 of each), so that y is off by its own rounding.
 */
size_t ssd_kv8_decode_workspace_bytes(const ssd_attn_cache* dims);

int ssd_kv8_decode(const ssd_attn_cache* dims, const ssd_kv8_pages* pages, const void* q, const int32_t* block_table,
                   const int64_t* seq_lens, const float* slopes, const float* table, void* y, void* workspace,
                   size_t workspace_bytes, void* stream);

/*
 * The values that the pages stand for, in `dtype`, packed: row cu_seqlens[s] + i of k and v [tokens, Hk, D] is position i
 * of sequence s, for ssd_attn_forward over what is cached.  Rows whose position is past seq_lens[s], outside the block table
 * or on no page are zeros; rows of no sequence are not written.
 *   cu_seqlens  DEVICE memory, nseq + 1 int64 offsets of the output rows, or NULL: tokens / nseq rows for each.
 */
int ssd_kv8_read(const ssd_attn_cache* dims, const ssd_kv8_pages* pages, int64_t tokens, const int64_t* cu_seqlens,
                 const int64_t* seq_lens, const int32_t* block_table, void* k, void* v, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSD_KV8_H */
