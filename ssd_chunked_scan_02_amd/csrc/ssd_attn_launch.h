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
};

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
    int q_slots, k_slots; // tiles of the packed axes (bounds: some are empty)
    float scale, cap;
    AttnBuckets bk;
};

// 0 on success, -1 when HIP rejects a launch, -2 for an unsupported shape.
int launch_attn_forward(const AttnParams& p, int dtype, int D, int bias, hipStream_t stream);
int launch_attn_backward(const AttnParams& p, int dtype, int D, int bias, hipStream_t stream);

}  // namespace ssd
