// Device helpers of the rotation and of the append to the 8-bit cache: a token's place in its sequence, its angles, and
// sixteen bytes of a head rotated.  gfx950 only.
#pragma once

#include "ssd_attn_common.h"

namespace ssd {
namespace attn {

// A token for each workgroup; more of them than a row of the grid holds go on in its next row.
constexpr int kTokenRow = 1 << 22;
inline dim3 token_grid(int64_t tokens) {
    return dim3((unsigned)(tokens < kTokenRow ? tokens : kTokenRow), (unsigned)((tokens + kTokenRow - 1) / kTokenRow));
}

// Angle pos * inv_freq of a pair, as turns of pi reduced in fp64: pos * inv_freq is exact to 53 bits there, and a far
// position's turns leave an fp32 no fraction.
__device__ __forceinline__ double half_turns(int64_t pos, float inv_freq) {
    const double turns = (double)pos * (double)inv_freq * 0.15915494309189535;
    return 2.0 * (turns - rint(turns));
}

// E elements of a head from its element `d` on (x), rotated in fp32 by the sines and cosines of its pairs; partner: the
// other elements of the pairs where they lie apart.  Each product is rounded by itself.
template <typename T, int E, typename V>
__device__ __forceinline__ void rotate(const V& x, const V& partner, int d, int rot, int interleaved, const float* cs, const float* sn,
                                       float (&y)[E]) {
#pragma clang fp contract(off)
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float c = cs[(d + e) / 2], s = sn[(d + e) / 2], a = (float)x[e], b = (float)x[e + 1];
            y[e] = a * c - b * s;
            y[e + 1] = b * c + a * s;
        }
    } else if (d < rot) {
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = (float)x[e] * cs[d + e] - (float)partner[e] * sn[d + e];
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = (float)x[e] * cs[d - rot + e] + (float)partner[e] * sn[d - rot + e];
    }
}

}  // namespace attn
}  // namespace ssd
