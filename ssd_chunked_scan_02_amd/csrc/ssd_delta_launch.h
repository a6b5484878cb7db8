// Host-side launch interface of the gated delta rule (ssd_delta*.hip), between the C ABI (ssd_delta_api.cpp) and its
// kernels, and the layout of its workspace.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssd {

constexpr int kDeltaChunk = 64;  // tokens of a chunk
constexpr int kDeltaCols = 32;   // value dimensions come in multiples of these (a walk's workgroup takes 16 or 32 columns)

// Chunk c of the sequence that begins at token `lo` of the packed axis has slot lo / 64 + s + c: sequences of any
// lengths then have slots of their own, total / 64 + nseq of them at most.
inline int64_t delta_slots(int64_t total, int64_t nseq) { return total / kDeltaChunk + nseq; }

struct DeltaParams {
    const void* q;          // [total, G, N]
    const void* k;
    const void* v;          // [total, H, P]
    const float* log_a;     // [total, H]
    const float* beta;
    const int64_t* cu;      // null: nseq sequences of `each` tokens
    const float* init;      // [nseq, H, N, P] or null
    void* y;                // [total, H, P]
    float* final_state;     // or null
    // backward
    const void* dy;
    const float* dfinal;    // or null
    void* dq;
    void* dk;
    void* dv;
    float* dlog_a;
    float* dbeta;
    float* dinit;           // or null
    // workspace, by slot and head (group): operands of the walks in the order that their lanes load them
    void* z;                // [slots, H][terms][64 x 64]: Z, rows by tile
    void* scores;           // [slots, H][terms][64 x 64]: decayed q . k
    void* zt;               // their transposes (backward)
    void* scores_t;
    void* kr;               // [slots, G][64 x N]: rows of K and Q by tile, zeros behind a sequence's end
    void* qr;
    float* gates;           // [slots, H][kDeltaGates][64]
    float* states;          // [slots + nseq, H, N, P]: the state before each chunk, and after the last
    float* wrong;           // [total, H, P]: e
    void* dstates;          // [slots, H, N, P]: gradient of the state after each chunk
    void* dstates_rest;     // bf16: what its rounding leaves, and (below) that of dv, rounded: the second terms of operands
    void* dv_rest;          // [total, H, P]
    float* dot_y;           // [slots, H, P / cols][64]: dy . y of a workgroup's columns
    float* dot_v;           // dv . v
    float* dot_b;           // x . e
    float* dot_s;           // [slots, H, P / cols][4]: <dstate, state> after each chunk
    float* dot_0;           // [nseq, H, P / cols][4]: before the first, where there is an init
    int64_t nseq, total, each, slots;
    int64_t q_stride, k_stride, v_stride;  // elements from one token to the next
    int H, G, N, P;
    int cols;               // columns of the state of a walk's workgroup: 16 or 32
    float scale;
};

// rows of `gates`: e^g, e^(g of the chunk's end - g), beta, and g in two parts
enum { kGateIn = 0, kGateOut = 1, kGateBeta = 2, kGateHigh = 3, kGateLow = 4, kDeltaGates = 5 };

struct DeltaStepParams {
    float* state;  // [nseq, H, N, P]
    const void* q;
    const void* k;
    const void* v;
    const float* log_a;
    const float* beta;
    void* y;
    int64_t nseq, q_stride, k_stride, v_stride;
    int H, G, N, P;
    float scale;
};

// 0 on success, -1 when HIP rejects a launch, -2 for an unsupported shape.
int launch_delta_forward(const DeltaParams& p, int dtype, hipStream_t stream);
int launch_delta_backward(const DeltaParams& p, int dtype, hipStream_t stream);
int launch_delta_step(const DeltaStepParams& p, int dtype, hipStream_t stream);

}  // namespace ssd
