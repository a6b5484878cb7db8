// Attention over a packed batch of documents, forward, gfx950:
//     s_ij = scale q_i.k_j, capped to c tanh(s / c), plus a bias by distance;  p = softmax over the
//     visible j;  y_i = sum_j p_ij v_j;  lse_i = log sum_j exp s_ij.
//
// One pass over the keys with a running maximum m and sum l (in log2 units): a workgroup of four waves
// owns 128 queries of one head and document, 32 a wave, and streams 64-key tiles (32 in fp32) through
// LDS, double buffered, the next tile's global loads in flight while the present one is used.  A wave
// forms S^T = K Q^T (queries in lanes), so m and l are one number a lane, and P^T in its accumulator
// layout is the operand of O^T += V^T P^T (ssd_attn_common.h).  O is rescaled only when a row's maximum
// has grown by more than 2^8: weights are relative to m, so a late m costs no accuracy.
#include "ssd_attn_common.h"

namespace ssd {
namespace attn {
namespace {

constexpr float kLazy = 8.f;  // log2 growth of a maximum that is let pass without a rescale

template <typename T, int D, bool CAP, int BIAS>
__global__ void __launch_bounds__(kThreads, 2) attn_fwd_kernel(AttnParams p) {
    using O = Op<T>;
    using L = Tile<T, D>;
    using Frag = typename O::Frag;
    constexpr int KT = O::kKT, NS = KT / 32, NT = D / O::kK, DT = D / 32, PK = 32 / O::kK;
    __shared__ __attribute__((aligned(16))) T ks[2][L::kElems];
    __shared__ __attribute__((aligned(16))) T vs[2][L::kElems];
    __shared__ float lut[BIAS == kBiasBuckets ? 2 * kMaxDistance + 1 : 1];

    int slot, head;
    work_item(blockIdx.x, p.q_slots, p.H, slot, head);
    const Span sp = find_span(p, slot, false);
    if (sp.tile < 0) return;
    const int kvh = head / (p.H / p.Hk);
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, half = lane / 32;
    const int shift = sp.lk - sp.lq;  // position of query 0 on the key axis
    int prefix = 0;
    if (p.prefix) prefix = (int)clamp64(p.prefix[sp.seq], 0, sp.lk);

    // keys [0, limit(i)) are visible to query i
    auto limit = [&](int i) { return p.causal ? max(min(max(i + shift + 1, prefix), sp.lk), 0) : sp.lk; };
    const int row0 = sp.tile * kBM + wave * 32, row = row0 + lane % 32;
    const int wg_limit = limit(min(sp.tile * kBM + kBM, sp.lq) - 1);
    const int ntiles = (wg_limit + KT - 1) / KT;
    const int my_limit = row < sp.lq ? limit(row) : 0;
    const int wave_most = row0 < sp.lq ? limit(min(row0 + 32, sp.lq) - 1) : 0;  // any query of the wave
    const int wave_least = limit(row0);                                         // every query of the wave

    const T* kg = static_cast<const T*>(p.k) + sp.k0 * p.k_stride + (int64_t)kvh * D;
    const T* vg = static_cast<const T*>(p.v) + sp.k0 * p.v_stride + (int64_t)kvh * D;

    Frag qf[NT];
    {
        const T* qg = static_cast<const T*>(p.q) + (sp.q0 + min(row, sp.lq - 1)) * p.q_stride + (int64_t)head * D;
#pragma unroll
        for (int t = 0; t < NT; ++t) qf[t] = __builtin_bit_cast(Frag, ld16(qg + (2 * t + half) * O::kE));
    }
    uint4 kb[L::kLoads], vb[L::kLoads];
    if (ntiles > 0) {
        L::load(kb, kg, p.k_stride, 0, sp.lk - 1);
        L::load(vb, vg, p.v_stride, 0, sp.lk - 1);
    }
    Score sc;
    sc.init(p.scale, p.cap, CAP, sizeof(T) == 4);
    float slope2 = 0.f;
    if constexpr (BIAS == kBiasSlopes) slope2 = p.slopes[head] * kLog2e;
    if constexpr (BIAS == kBiasBuckets) fill_bias(lut, p, head);
    if (ntiles > 0) {
        L::store(ks[0], kb);
        L::store(vs[0], vb);
    }
    __syncthreads();

    f32x16 o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = f32x16{};
    float m = kNoMax, l = 0.f;  // l: this lane half's share
    const int qpos = row + shift;

    for (int t = 0; t < ntiles; ++t) {
        const int k0 = t * KT;
        if (t + 1 < ntiles) {
            L::load(kb, kg, p.k_stride, k0 + KT, sp.lk - 1);
            L::load(vb, vg, p.v_stride, k0 + KT, sp.lk - 1);
        }
        const T* kt = ks[t & 1];
        const T* vt = vs[t & 1];
        if (k0 < wave_most) {
            f32x16 s[NS];
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                s[n] = f32x16{};
#pragma unroll
                for (int i = 0; i < NT; ++i) s[n] = O::mma(L::rows(kt, 32 * n, i, lane), qf[i], s[n]);
            }
            // scores in log2 units
            const int rel0 = k0 + 4 * half - qpos;  // relative position of register 0 of sub-tile 0
            if constexpr (CAP) {
#pragma unroll
                for (int n = 0; n < NS; ++n)
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[n][r] = sc.c2 * sc.template tanh_of<T>(s[n][r]);
            }
            const float a = CAP ? 1.f : sc.a;
            if constexpr (BIAS == kBiasNone) {
                if constexpr (!CAP) {
#pragma unroll
                    for (int n = 0; n < NS; ++n) s[n] *= a;
                }
            } else if constexpr (BIAS == kBiasSlopes) {
                const float rel = (float)rel0;
#pragma unroll
                for (int n = 0; n < NS; ++n)
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[n][r] = s[n][r] * a - slope2 * fabsf(rel + (float)(32 * n + acc_row(r)));
            } else {
                const int md = p.bk.max_distance;
                const int lowest = k0 - (row0 + 31 + shift), highest = k0 + KT - 1 - (row0 + shift);
                if (highest <= -md || lowest >= md) {
                    const float b = lut[highest <= -md ? 0 : 2 * md];
#pragma unroll
                    for (int n = 0; n < NS; ++n)
#pragma unroll
                        for (int r = 0; r < 16; ++r) s[n][r] = s[n][r] * a + b;
                } else {
#pragma unroll
                    for (int n = 0; n < NS; ++n)
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            s[n][r] = s[n][r] * a + lut[min(max(rel0 + 32 * n + acc_row(r), -md), md) + md];
                }
            }
            if (k0 + KT > wave_least) {
                const int left = my_limit - k0 - 4 * half;
#pragma unroll
                for (int n = 0; n < NS; ++n)
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[n][r] = 32 * n + acc_row(r) < left ? s[n][r] : -INFINITY;
            }
            float mx = s[0][0];
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[n][r]);
            mx = fmaxf(mx, other_half(mx));
            if (__any(mx > m + kLazy)) {
                const float next = fmaxf(m, mx), keep = exp2_hw(m - next);
                m = next;
                l *= keep;
#pragma unroll
                for (int d = 0; d < DT; ++d) o[d] *= keep;
            }
            float add = 0.f;
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    s[n][r] = exp2_hw(s[n][r] - m);
                    add += s[n][r];
                }
            l += add;
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int kk = 0; kk < PK; ++kk) {
                    const Frag pf = O::pack(s[n], kk);
#pragma unroll
                    for (int d = 0; d < DT; ++d) o[d] = O::mma(L::cols(vt, 32 * n, kk, 32 * d, lane), pf, o[d]);
                }
        }
        if (t + 1 < ntiles) {
            L::store(ks[(t + 1) & 1], kb);
            L::store(vs[(t + 1) & 1], vb);
        }
        lds_barrier();
    }

    l += other_half(l);
    if (row >= sp.lq) return;
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // (an empty row is zero; a NaN stays one)
    T* yg = static_cast<T*>(p.y) + ((sp.q0 + row) * p.H + head) * D;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int r = 0; r < 16; r += 4)
            store4(yg + 32 * d + 2 * r + 4 * half, o[d][r] * inv, o[d][r + 1] * inv, o[d][r + 2] * inv, o[d][r + 3] * inv);
    if (p.lse && half == 0) p.lse[(sp.q0 + row) * p.H + head] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
}

template <typename T, int D, bool CAP, int BIAS>
int launch_fwd(const AttnParams& p, hipStream_t stream) {
    const int64_t grid = (int64_t)p.q_slots * p.H;
    if (grid == 0) return 0;
    hipLaunchKernelGGL((attn_fwd_kernel<T, D, CAP, BIAS>), dim3((unsigned)grid), dim3(kThreads), 0, stream, p);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}
template <typename T, int D, bool CAP>
int launch_fwd(const AttnParams& p, int bias, hipStream_t stream) {
    switch (bias) {
        case kBiasNone: return launch_fwd<T, D, CAP, kBiasNone>(p, stream);
        case kBiasSlopes: return launch_fwd<T, D, CAP, kBiasSlopes>(p, stream);
        default: return launch_fwd<T, D, CAP, kBiasBuckets>(p, stream);
    }
}
template <typename T>
int launch_fwd(const AttnParams& p, int D, int bias, hipStream_t stream) {
    const bool cap = p.cap > 0.f;
    switch (D) {
        case 32: return cap ? launch_fwd<T, 32, true>(p, bias, stream) : launch_fwd<T, 32, false>(p, bias, stream);
        case 64: return cap ? launch_fwd<T, 64, true>(p, bias, stream) : launch_fwd<T, 64, false>(p, bias, stream);
        case 128: return cap ? launch_fwd<T, 128, true>(p, bias, stream) : launch_fwd<T, 128, false>(p, bias, stream);
        default: return -2;
    }
}

}  // namespace
}  // namespace attn

int launch_attn_forward(const AttnParams& in, int dtype, int D, int bias, hipStream_t stream) {
    AttnParams p = in;
    p.q_slots = (int)attn::slots_of(p.cu_q, p.total_q, p.nseq);
    return dtype == 1 ? attn::launch_fwd<__bf16>(p, D, bias, stream) : attn::launch_fwd<float>(p, D, bias, stream);
}

}  // namespace ssd
