// Host-side launch interface of the 8-bit paged cache (ssd_kv8.hip) and of the rotation (ssd_rotary.hip), between the C ABI
// (ssd_kv8_api.cpp) and their kernels.
#pragma once

#include "ssd_attn_launch.h"

namespace ssd {

struct Kv8Pages {
    uint8_t* k;       // [num_pages, page_size, Hk, D]
    uint8_t* v;
    float* k_scale;   // [num_pages, page_size, Hk]
    float* v_scale;
};

struct Kv8ReadParams {
    Kv8Pages pages;
    const int* block_table;
    const int64_t* seq_lens;
    const int64_t* cu;  // null: `each` rows of a sequence
    void* k;            // [tokens, Hk, D]
    void* v;
    int64_t nseq, tokens, each;
    int Hk, D, num_pages, page_size, max_pages;
};

struct RotateParams {
    const void* q;
    const void* k;      // null: no keys
    void* q_out;
    void* k_out;
    const int64_t* cu;  // null: `each` tokens of a sequence
    const int64_t* start;
    const float* inv_freq;
    int64_t nseq, total, each, q_stride, k_stride;
    int H, Hk, D, rot, interleaved;
    float magnitude, sign;  // of the angle
};

// The decode step takes its parameters as ssd_attn_decode, and its caches from the pages.
// 0 on success, -1 when HIP rejects a launch, -2 for an unsupported shape.
int launch_kv8_append(const AppendParams& p, const Kv8Pages& pages, int dtype, int format, hipStream_t stream);
int launch_kv8_decode(const DecodeParams& p, const Kv8Pages& pages, int dtype, int format, int D, int bias, hipStream_t stream);
int launch_kv8_read(const Kv8ReadParams& p, int dtype, int format, hipStream_t stream);
int launch_rotate(const RotateParams& p, int dtype, hipStream_t stream);

}  // namespace ssd
