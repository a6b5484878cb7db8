// attn_join_kernel: y of one query per sequence from the parts of its split keys (of ssd_attn_decode.hip and ssd_kv8.hip).
#pragma once

#include "ssd_attn_common.h"

namespace ssd {
namespace attn {
namespace {

// y of one (sequence, head) from its splits; a workgroup takes kThreads / (D / 4) of them.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) attn_join_kernel(DecodeParams p, int64_t units) {
    constexpr int PER = D / 4;
    const int64_t at = (int64_t)blockIdx.x * (kThreads / PER) + threadIdx.x / PER;
    if (at >= units) return;
    const int d = 4 * (int)(threadIdx.x % PER);
    const float* ml = p.part_ml + at * p.splits * 2;
    float top = kNoMax;
    for (int i = 0; i < p.splits; ++i) top = fmaxf(top, ml[2 * i]);
    float sum = 0.f;
    f32x4 v{};
    for (int i = 0; i < p.splits; ++i) {
        const float f = exp2_hw(ml[2 * i] - top);
        sum += f * ml[2 * i + 1];
        v += f * as_f32x4(ld16(p.part_o + (at * p.splits + i) * D + d));
    }
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    store4(static_cast<T*>(p.y) + at * D + d, v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
}

template <typename T, int D>
int launch_join(const DecodeParams& p, hipStream_t stream) {
    const int64_t units = p.nseq * p.H;
    const int per = kThreads / (D / 4);
    hipLaunchKernelGGL((attn_join_kernel<T, D>), dim3((unsigned)((units + per - 1) / per)), dim3(kThreads), 0, stream, p, units);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace
}  // namespace attn
}  // namespace ssd
