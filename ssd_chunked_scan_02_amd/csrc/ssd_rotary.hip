// Rotary positions of queries and keys, gfx950.
//
// A token's angles are the same for all of its heads: a workgroup takes one token, has each angle's sine and cosine taken once
// (reduced in fp64, taken in fp32) and rotates the heads by them, sixteen bytes a thread.  Bound by memory: 16385 tokens, 32/8 heads of 128, bf16, 71 us, 4.7 TB/s.
#include "ssd_kv8_launch.h"
#include "ssd_rotary_common.h"

namespace ssd {
namespace attn {
namespace {

template <typename T>
__global__ void __launch_bounds__(kThreads) rotate_kernel(RotateParams p) {
    constexpr int E = 16 / (int)sizeof(T);
    typedef T vec __attribute__((ext_vector_type(E)));
    __shared__ float cs[kMaxRot], sn[kMaxRot];
    const int64_t tok = (int64_t)blockIdx.y * kTokenRow + blockIdx.x;
    if (tok >= p.total) return;
    int64_t s, first;
    if (p.cu) {
        s = last_at_most((int)p.nseq, [&](int i) { return p.cu[i] <= tok; });
        first = p.cu[s];
        if (tok < first || tok >= p.cu[s + 1]) return;  // a token of no sequence
    } else {
        s = tok / p.each;
        first = s * p.each;
    }
    const int64_t pos = tok - first + (p.start ? p.start[s] : 0);
    for (int i = threadIdx.x; i < p.rot; i += kThreads) {
        float a, b;
        sincospif((float)half_turns(pos, p.inv_freq[i]), &a, &b);
        cs[i] = p.magnitude * b;
        sn[i] = p.sign * p.magnitude * a;
    }
    __syncthreads();
    const int CH = p.D / E, qc = p.H * CH, total = qc + (p.k ? p.Hk * CH : 0);
    for (int i = threadIdx.x; i < total; i += kThreads) {
        const bool q = i < qc;
        const int at = q ? i : i - qc, d = (at % CH) * E;
        const T* in = q ? static_cast<const T*>(p.q) + tok * p.q_stride : static_cast<const T*>(p.k) + tok * p.k_stride;
        T* out = q ? static_cast<T*>(p.q_out) + tok * p.H * p.D : static_cast<T*>(p.k_out) + tok * p.Hk * p.D;
        vec x = __builtin_bit_cast(vec, ld16(in + at * E));
        if (d < 2 * p.rot) {
            const int over = p.interleaved ? 0 : d < p.rot ? p.rot : -p.rot;
            const vec z = __builtin_bit_cast(vec, ld16(in + at * E + over));
            float y[E];
            rotate<T, E>(x, z, d, p.rot, p.interleaved, cs, sn, y);
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = (T)y[e];
        }
        st16(out + at * E, __builtin_bit_cast(uint4, x));
    }
}

}  // namespace
}  // namespace attn

int launch_rotate(const RotateParams& p, int dtype, hipStream_t stream) {
    const dim3 grid = attn::token_grid(p.total);
    if (dtype == 1) hipLaunchKernelGGL(attn::rotate_kernel<__bf16>, grid, dim3(kThreads), 0, stream, p);
    else hipLaunchKernelGGL(attn::rotate_kernel<float>, grid, dim3(kThreads), 0, stream, p);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace ssd
