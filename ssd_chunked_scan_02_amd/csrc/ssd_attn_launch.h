// Host-side launch interface of the attention operators (ssd_attn*.hip), between the C ABI
// (ssd_attn_api.cpp) and their kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssd {

// Bias of a score by the distance between its query and its key.
enum AttnBias { kBiasNone = 0, kBiasSlopes = 1, kBiasBuckets = 2 };

// Buckets of key position minus query position.  Within a direction the bucket of distance d is the
// number of borders at most d; with `both` directions, keys behind the query (rel > 0) take the
// second half of the table.  Distances of max_distance and more share the last bucket.
constexpr int kMaxBorders = 64;
constexpr int kMaxDistance = 1024;
struct AttnBuckets {
    int total;         // buckets in the table
    int both;          // 1: two directions
    int max_distance;  // >= every border
    int nborders;      // buckets of one direction - 1
    int borders[kMaxBorders];
    uint8_t of[kMaxDistance + 1];  // a direction's bucket by distance, to max_distance
};

// Workgroups of 128 rows below which the four waves of one split instead (kOwn in ssd_attn_common.h), by the
// bytes of a row.  A split workgroup's tiles take most of a CU's LDS from rows of 256 bytes on, so that it
// stays alone there, and half of it below.  bf16, causal, one sequence, forward / dq / dk and dv in us,
// split against not:
//     64 wide, 4096 tokens   256 workgroups 48 / 57 / 64 against 68 / 96 / 112, 512: 88 / 101 / 123 against 73 / 105 / 120
//     64 wide, 1024 tokens   256: 22 / 25 / 29 against 22 / 30 / 34, 512: 39 / 46 / 53 against 24 / 35 / 39
//     128 wide, 4096 tokens  128: 52 / 58 / 68 against 85 / 113 / 129, 256: 99 / 110 / 129 against 87 / 120 / 136
//     128 wide, 1024 tokens  128: 23 / 27 / 29 against 26 / 37 / 38, 256: 45 / 52 / 57 against 28 / 42 / 42
// (In fp32 both widths would gain from splitting at 256 still: 64 wide, 1024 tokens, 68 / 90 / 112 against 83 / 115 / 157.)
inline int64_t attn_split_below(int row_bytes) { return row_bytes >= 256 ? 256 : 384; }
// HIP counts the threads of a launch in 32 bits; calls past that are refused before their first launch.
inline bool launchable(int64_t groups, int threads) { return groups * threads < ((int64_t)1 << 32); }
// Tiles of a packed axis, at most: its whole tiles, and one more for each sequence.
inline int64_t attn_slots(const int64_t* cu, int64_t total, int64_t nseq, int own) {
    if (nseq == 0) return 0;
    return cu ? total / own + nseq : nseq * ((total / nseq + own - 1) / own);
}
// Key gradients of a small problem: parts of a tile's queries, so that the workgroups reach the 256 CUs twice.
inline int attn_key_parts(const int64_t* cu_k, int64_t total_k, int64_t nseq, int64_t Hk, int row_bytes) {
    if (attn_slots(cu_k, total_k, nseq, 128) * Hk >= attn_split_below(row_bytes)) return 1;
    const int64_t grid = attn_slots(cu_k, total_k, nseq, 32) * Hk, n = grid > 0 ? 512 / grid : 1;
    return n < 1 ? 1 : n > 8 ? 8 : (int)n;
}

struct AttnParams {
    const void* q;
    const void* k;
    const void* v;
    const void* dy;
    const float* slopes;  // [H]
    const float* table;   // [buckets, H]
    const int64_t* cu_q;  // null: nseq equal sequences
    const int64_t* cu_k;  // null: nseq equal sequences
    const int64_t* prefix;
    void* y;              // forward: output; backward: input
    float* lse;           // [total_q, H]; forward: output (may be null); backward: input
    void* dq;
    void* dk;
    void* dv;
    float* dtable;
    float* delta;         // workspace [total_q, H]
    float* table_part;    // workspace [query slots * H, buckets]
    int64_t nseq, total_q, total_k;
    int64_t q_stride, k_stride, v_stride;  // elements from one token to the next
    int H, Hk;
    int causal;
    int pack;             // query heads of a group that share the rows of a query tile (see Rows), or 1
    int q_slots, k_slots; // tiles of the packed axes (bounds: some are empty)
    int each_q, each_k, each_q_tiles, each_k_tiles;  // equal sequences: their lengths and tiles
    int parts;            // key gradients: workgroups that share one tile's queries (1: none)
    float* dkv_part;      // workspace [2][parts, total_k, Hk, D], or null
    int2* plan_q;         // workspace: (sequence, tile) of the slots in order of their work, or null
    int2* plan_k;
    float scale, cap;
    AttnBuckets bk;
};

// One query per sequence over a paged cache.
struct DecodeParams {
    const void* q;            // [nseq, H, D]
    const void* k_cache;      // [num_pages, page_size, Hk, D]
    const void* v_cache;
    const int* block_table;   // [nseq, max_pages]
    const int64_t* seq_lens;  // [nseq]
    const float* slopes;
    const float* table;
    void* y;                  // [nseq, H, D]
    float* part_o;            // workspace [nseq, H, splits, D]
    float* part_ml;           // workspace [nseq, H, splits, 2]
    int64_t nseq, q_stride;
    int H, Hk, num_pages, page_size, max_pages, splits;
    int wide;                 // 1: eight waves a workgroup instead of four
    float scale, cap;
    AttnBuckets bk;
};

// Tokens appended to a paged cache, rotated by their positions.
constexpr int kMaxRot = 64;
struct AppendParams {
    const void* q;  // null: no queries
    const void* k;
    const void* v;
    void* q_out;
    void* k_cache;
    void* v_cache;
    const int* block_table;
    const int64_t* seq_lens;  // lengths with the new tokens
    const int64_t* cu;        // null: one token per sequence
    const float* inv_freq;    // [rot]
    int64_t nseq, tokens, q_stride, k_stride, v_stride;
    int H, Hk, D, num_pages, page_size, max_pages;
    int rot;                  // pairs that are rotated
    int interleaved;
};

// 0 on success, -1 when HIP rejects a launch, -2 for an unsupported shape.
int launch_attn_forward(const AttnParams& p, int dtype, int D, int bias, hipStream_t stream);
int launch_attn_backward(const AttnParams& p, int dtype, int D, int bias, hipStream_t stream);
int launch_attn_decode(const DecodeParams& p, int dtype, int D, int bias, hipStream_t stream);
int launch_kv_append(const AppendParams& p, int dtype, hipStream_t stream);

}  // namespace ssd
