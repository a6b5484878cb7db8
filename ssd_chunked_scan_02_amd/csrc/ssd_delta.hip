// The gated delta rule, forward: the chunked scan and the single-token step, gfx950.
//
//     S~ = a_t S_{t-1},   e_t = v_t - S~^T k_t,   S_t = S~ + k_t (beta_t e_t)^T,   y_t = scale S_t^T q_t
#include "ssd_delta_prep.h"
#include "ssd_delta_walk.h"

namespace ssd {
namespace delta {
namespace {

// One token: a workgroup takes 32 columns of one state, a thread four of them in every 32nd row.  Both products with
// the old state are taken in the one pass that reads it: S_t^T q = a S^T q + (k.q) beta e.  Bound by the state's bytes, read
// once and written once: 64 sequences, 32 heads of 128 by 128, 52 us, 5.1 TB/s (41 us where its states are still in the last-level cache);
// one sequence 13 us, the host's call.
template <typename T, int N>
__global__ void __launch_bounds__(kThreads) delta_step_kernel(DeltaStepParams p) {
    constexpr int R = N / 32;
    __shared__ float part[kWaves][8][9];
    const int blocks = p.P / kDeltaCols, cb = (int)(blockIdx.x % blocks);
    const int64_t sh = blockIdx.x / blocks, s = sh / p.H;
    const int h = (int)(sh % p.H), grp = h / (p.H / p.G), c4 = threadIdx.x % 8, rg = threadIdx.x / 8;
    const T* kp = static_cast<const T*>(p.k) + s * p.k_stride + grp * N;
    const T* qp = static_cast<const T*>(p.q) + s * p.q_stride + grp * N;
    float* state = p.state + (sh * N) * p.P + cb * kDeltaCols + 4 * c4;
    const float a = expf(p.log_a[sh]), beta = p.beta[sh];
    f32x4 x[R];
    float k[R];
    f32x4 ks{}, qs{};
    float kq = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int n = rg + 32 * i;
        x[i] = as_f32x4(ld16(state + (int64_t)n * p.P));
        k[i] = to_f32(kp[n]);
        const float q = to_f32(qp[n]);
        ks += k[i] * x[i];
        qs += q * x[i];
        kq += k[i] * q;
    }
#pragma unroll
    for (int off = 8; off < kWave; off <<= 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            ks[e] += __shfl_xor(ks[e], off, kWave);
            qs[e] += __shfl_xor(qs[e], off, kWave);
        }
        kq += __shfl_xor(kq, off, kWave);
    }
    if (threadIdx.x % kWave < 8) {
        float* to = part[threadIdx.x / kWave][c4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            to[e] = ks[e];
            to[4 + e] = qs[e];
        }
        to[8] = kq;
    }
    __syncthreads();
    ks = qs = f32x4{};
    kq = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            ks[e] += part[w][c4][e];
            qs[e] += part[w][c4][4 + e];
        }
        kq += part[w][c4][8];
    }
    const int64_t col = (int64_t)h * p.P + cb * kDeltaCols + 4 * c4;
    const T* vp = static_cast<const T*>(p.v) + s * p.v_stride + col;
    f32x4 u;
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = beta * (to_f32(vp[e]) - a * ks[e]);
#pragma unroll
    for (int i = 0; i < R; ++i) st16(state + (int64_t)(rg + 32 * i) * p.P, __builtin_bit_cast(uint4, a * x[i] + k[i] * u));
    if (rg == 0) {
        const f32x4 y = p.scale * (a * qs + kq * u);
        store4(static_cast<T*>(p.y) + s * p.H * p.P + col, y[0], y[1], y[2], y[3]);
    }
}

template <typename T, int N>
int launch_step(const DeltaStepParams& p, hipStream_t stream) {
    hipLaunchKernelGGL((delta_step_kernel<T, N>), dim3((unsigned)(p.nseq * p.H * (p.P / kDeltaCols))), dim3(kThreads), 0, stream, p);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

template <typename T, int N>
int launch_forward(const DeltaParams& p, hipStream_t stream) {
    if (p.slots > 0 && p.total > 0) {
        const int rc = launch_prep<T, N, false>(p, stream);
        if (rc != 0) return rc;
    }
    return launch_walk<T, N, false>(p, stream);
}

}  // namespace
}  // namespace delta

int launch_delta_forward(const DeltaParams& p, int dtype, hipStream_t stream) {
    switch (p.N) {
        case 32: return dtype == 1 ? delta::launch_forward<__bf16, 32>(p, stream) : delta::launch_forward<float, 32>(p, stream);
        case 64: return dtype == 1 ? delta::launch_forward<__bf16, 64>(p, stream) : delta::launch_forward<float, 64>(p, stream);
        case 128: return dtype == 1 ? delta::launch_forward<__bf16, 128>(p, stream) : delta::launch_forward<float, 128>(p, stream);
        default: return -2;
    }
}

int launch_delta_step(const DeltaStepParams& p, int dtype, hipStream_t stream) {
    switch (p.N) {
        case 32: return dtype == 1 ? delta::launch_step<__bf16, 32>(p, stream) : delta::launch_step<float, 32>(p, stream);
        case 64: return dtype == 1 ? delta::launch_step<__bf16, 64>(p, stream) : delta::launch_step<float, 64>(p, stream);
        case 128: return dtype == 1 ? delta::launch_step<__bf16, 128>(p, stream) : delta::launch_step<float, 128>(p, stream);
        default: return -2;
    }
}

}  // namespace ssd
