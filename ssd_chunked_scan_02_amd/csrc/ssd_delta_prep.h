// delta_prep_kernel: what the walks of the gated delta rule need of each chunk of 64 tokens, all chunks at once.
//
// With g_i the running sum of log a in the chunk, D_ij = e^(g_i - g_j), L_ij = D_ij k_i.k_j (j < i) and B = diag(beta):
//     Z = -(I + L B)^-1 L,   so that  E = (I + L B)^-1 R = R + Z B R   and   (I + B L)^-T dU = dU + Z^T B dU,
// which is finite for any beta, zero among them.  A workgroup takes one chunk and key head: K K^T and Q K^T once on
// the matrix unit (exact products, fp32 sums), then for each value head of the group the decays, Z by blocks of 16
// (substitution on the diagonal, fp32 MFMA products beside it) and the decayed scores, stored as operands.
// g is kept in two fp32 parts, so that differences of far sums keep their bits; decays below e^-160 are taken as that,
// which is zero in fp32 in every product.
//
// Bound by bytes, most of them written: Z in three terms and the scores in two are 30 KB a chunk and value head in bf16, and 72 KB in the
// backward pass (three terms of the scores, and both transposed), in places of 40 and 96 with the steps that are zero throughout; the
// rows of K and Q once more.  8 x 2048 tokens, 24 heads of 128 by 64, bf16: 113 us, 227 MB read and 398 written (5.5 TB/s); in the backward
// pass 154 us, 227 and 662 MB (5.8 TB/s); 16384 tokens, 32/16 heads of 128 by 128: 113 us, 564 MB.  All chunks
// at once here leaves the walks a chain without the substitution; a walk that made its own Z would do so in each of its
// workgroups (4 to 16 of a head).
#pragma once

#include "ssd_delta_common.h"

namespace ssd {
namespace delta {

constexpr int kLdz = kC + 4;  // LDS row stride of a 64 x 64 fp32 matrix

// Operand fragments of a lower triangular [64][64] matrix of LDS, or of its transpose, to memory: rows by tile, then steps,
// then lanes.  Steps that are zero throughout have their places and are not written (nor read).
template <typename T, bool TRANSPOSED, int TERMS>
__device__ __forceinline__ void emit(T* out, const float* at) {
    using M = Mat<T>;
    constexpr int KC = kC / M::kK, TILES = M::kK / 16;
    for (int f = threadIdx.x; f < 4 * KC * kWave; f += kThreads) {
        const int lane = f % kWave, ks = f / kWave % KC, rt = f / (kWave * KC), m = lane % 16, g = lane / 16;
        float x[M::kE];
        if (TRANSPOSED ? TILES * ks + TILES - 1 < rt : TILES * ks > rt) continue;
#pragma unroll
        for (int i = 0; i < TILES; ++i) {  // a step is of one or two tiles, four tokens of each in a lane
            const int ct = TILES * ks + i;
            const bool left = TRANSPOSED ? ct >= rt : ct <= rt;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[4 * i + e] = !left ? 0.f : TRANSPOSED ? at[(16 * ct + 4 * g + e) * kLdz + 16 * rt + m] : at[(16 * rt + m) * kLdz + 16 * ct + 4 * g + e];
        }
        put_frag<TERMS>(out + (int64_t)f * M::kE, kC * kC, x);
    }
}

// A chunk's 64 rows of N elements, zeros from row `have` on, into LDS.
template <typename T, int N>
__device__ __forceinline__ void stage_rows(T* to, const T* from, int64_t stride, int have) {
    using M = Mat<T>;
    const Block rows = Chunks(from, have, stride, N).block(true);
    constexpr int CH = N / M::kE, PER = kC * CH / kThreads;
    typename M::Frag x[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        x[i] = rows.template frag<T>((uint32_t)(((threadIdx.x + i * kThreads) / CH * stride + (threadIdx.x + i * kThreads) % CH * M::kE) * sizeof(T)), 0);
#pragma unroll
    for (int i = 0; i < PER; ++i)
        st16(to + (threadIdx.x + i * kThreads) / CH * (N + M::kPad) + (threadIdx.x + i * kThreads) % CH * M::kE, __builtin_bit_cast(uint4, x[i]));
}

template <typename T, int N> constexpr int prep_lds_bytes() {
    const int rows = kC * (N + Mat<T>::kPad) * (int)sizeof(T), mats = 2 * kC * kLdz * 4;
    return rows > mats ? rows : mats;
}

template <typename T, int N, bool BACKWARD>
__global__ void __launch_bounds__(kThreads, 3) delta_prep_kernel(DeltaParams p) {
    using M = Mat<T>;
    using Frag = typename M::Frag;
    constexpr int KN = N / M::kK, TERMS = M::kTerms;
    __shared__ __attribute__((aligned(16))) char mem[prep_lds_bytes<T, N>()];
    __shared__ float ghi[kWaves][kC], glo[kWaves][kC], betas[kWaves][kC];  // of four heads at a time

    const int64_t slot = blockIdx.x / p.G;
    const int grp = blockIdx.x % p.G, group = p.H / p.G;
    const int64_t s = seq_of_slot(p, slot);
    const Span span = span_of(p, s);
    const int64_t chunk = slot - (span.lo / kC + s);
    if (chunk < 0 || chunk * kC >= span.len) return;
    const int64_t tok0 = span.lo + chunk * kC;
    const int have = (int)(span.len - chunk * kC < kC ? span.len - chunk * kC : kC);
    const int lane = threadIdx.x % kWave, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), m = lane % 16, g = lane / 16;

    // wave w's head of the next four: its gates, summed along the chunk
    float la = 0.f, be = 0.f;
    const auto load_gates = [&](int r) {
        const bool ok = r + w < group && lane < have;
        const int64_t tok = (tok0 + (ok ? lane : 0)) * p.H + grp * group + (ok ? r + w : 0);
        la = ok ? p.log_a[tok] : 0.f;
        be = ok ? p.beta[tok] : 0.f;
    };
    const auto put_gates = [&](int r) {
        if (r + w >= group) return;
        la = la < -160.f ? -160.f : la;
        double sum = la;
#pragma unroll
        for (int off = 1; off < kWave; off <<= 1) {
            const double o = __shfl_up(sum, off, kWave);
            if (lane >= off) sum += o;
        }
        const float hi = (float)sum, lo = (float)(sum - (double)hi);
        ghi[w][lane] = hi;
        glo[w][lane] = lo;
        betas[w][lane] = be;
        float* gates = p.gates + (slot * p.H + grp * group + r + w) * (kDeltaGates * kC) + lane;
        gates[kGateIn * kC] = expf(hi);
        gates[kGateOut * kC] = expf((float)(__shfl(sum, kWave - 1, kWave) - sum));
        gates[kGateBeta * kC] = be;
        gates[kGateHigh * kC] = hi;
        gates[kGateLow * kC] = lo;
    };
    load_gates(0);

    // k_i.k_j and q_i.k_j: wave w has rows 16 w .. of the lower tiles
    f32x4 kk[4], qk[4];
    {
        T* rows = reinterpret_cast<T*>(mem);
        const T* kp = static_cast<const T*>(p.k) + tok0 * p.k_stride + grp * N;
        const T* qp = static_cast<const T*>(p.q) + tok0 * p.q_stride + grp * N;
        Frag qf[KN];
        const Block qrows = Chunks(qp, have, p.q_stride, N).block(true);
        const uint32_t qat = (uint32_t)(((16 * w + m) * p.q_stride + g * M::kE) * sizeof(T));
#pragma unroll
        for (int t = 0; t < KN; ++t) qf[t] = qrows.frag<T>(qat, t * M::kK * sizeof(T));
        stage_rows<T, N>(rows, kp, p.k_stride, have);
        put_gates(0);
        __syncthreads();
        // the rows themselves, in the order of the walks' loads (as they lie in their tensors, a head's rows are often
        // some multiple of 4 KB apart, which are all of one channel of the L2)
        Frag kf[KN];
        const int64_t own = (slot * p.G + grp) * (int64_t)(N * kC) + (w * KN * kWave + lane) * M::kE;
#pragma unroll
        for (int t = 0; t < KN; ++t) {
            kf[t] = frag(rows + (16 * w + m) * (N + M::kPad) + t * M::kK + g * M::kE);
            st16(static_cast<T*>(p.kr) + own + t * (kWave * M::kE), __builtin_bit_cast(uint4, kf[t]));
            st16(static_cast<T*>(p.qr) + own + t * (kWave * M::kE), __builtin_bit_cast(uint4, qf[t]));
        }
#pragma unroll
        for (int ct = 0; ct < 4; ++ct) {
            kk[ct] = qk[ct] = f32x4{};
            if (ct > w) continue;
#pragma unroll
            for (int t = 0; t < KN; ++t) {
                const Frag kb = frag(rows + (16 * ct + m) * (N + M::kPad) + t * M::kK + g * M::kE);
                kk[ct] = M::mma(kf[t], kb, kk[ct]);
                qk[ct] = M::mma(qf[t], kb, qk[ct]);
            }
        }
        __syncthreads();
    }

    float* lm = reinterpret_cast<float*>(mem);  // L
    float* zm = lm + kC * kLdz;                 // the scores, then Z; tiles above the diagonal are not written
    for (int r = 0; r < group; ++r) {
        const int64_t at = slot * p.H + grp * group + r;
        if (r > 0 && r % kWaves == 0) {
            put_gates(r);
            __syncthreads();
        }
        if (r % kWaves == kWaves - 1) load_gates(r + 1);
        const float *const gh = ghi[r % kWaves], *const gl = glo[r % kWaves], *const beta = betas[r % kWaves];
#pragma unroll
        for (int ct = 0; ct < 4; ++ct) {
            if (ct > w) continue;
            const int j = 16 * ct + m;
            const float hj = gh[j], lj = gl[j];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 16 * w + 4 * g + e;
                const float d = j <= i ? expf((gh[i] - hj) + (gl[i] - lj)) : 0.f;
                lm[i * kLdz + j] = j < i ? d * kk[ct][e] : 0.f;
                zm[i * kLdz + j] = j <= i ? d * qk[ct][e] : 0.f;
            }
        }
        __syncthreads();
        constexpr int ST = terms_of_y<T>(BACKWARD);
        emit<T, false, ST>(static_cast<T*>(p.scores) + at * (ST * kC * kC), zm);
        if constexpr (BACKWARD) emit<T, true, TERMS>(static_cast<T*>(p.scores_t) + at * (TERMS * kC * kC), zm);

        // Z of the diagonal tile w, row by row: z_i = -L_i - sum_{j<i} L_ij beta_j z_j
        f32x4 z, inv;  // inv: row m, columns 4 g .. of (I + L B)^-1's diagonal tile, an operand
        {
            const float* lw = lm + (16 * w) * kLdz + 16 * w;
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = -lw[(4 * g + e) * kLdz + m];
#pragma unroll
            for (int i = 0; i < 15; ++i) {
                const float zi = beta[16 * w + i] * __shfl(z[i % 4], (i / 4) * 16 + m, kWave);
#pragma unroll
                for (int e = 0; e < 4; ++e) z[e] -= lw[(4 * g + e) * kLdz + i] * zi;
            }
            __syncthreads();  // (the scores are written)
#pragma unroll
            for (int e = 0; e < 4; ++e) zm[(16 * w + 4 * g + e) * kLdz + 16 * w + m] = z[e];
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = 4 * g + e;
            inv[e] = (m == c ? 1.f : 0.f) + zm[(16 * w + m) * kLdz + 16 * w + c] * beta[16 * w + c];
        }
        // Z of tile (w, w - d) = -inv (L + sum over the tiles k between, (L B)_wk Z_k)
#pragma unroll
        for (int d = 1; d < 4; ++d) {
            if (w >= d) {
                const int ct = w - d;
                f32x4 acc;
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] = lm[(16 * w + 4 * g + e) * kLdz + 16 * ct + m];
                for (int k = ct; k < w; ++k) {
                    const float* row = lm + (16 * w + m) * kLdz + 16 * k + 4 * g;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc = mfma_f32(row[e] * beta[16 * k + 4 * g + e], zm[(16 * k + 4 * g + e) * kLdz + 16 * ct + m], acc);
                }
                f32x4 out{};
#pragma unroll
                for (int e = 0; e < 4; ++e) out = mfma_f32(inv[e], acc[e], out);
#pragma unroll
                for (int e = 0; e < 4; ++e) zm[(16 * w + 4 * g + e) * kLdz + 16 * ct + m] = -out[e];
            }
            __syncthreads();
        }
        emit<T, false, TERMS>(static_cast<T*>(p.z) + at * (TERMS * kC * kC), zm);
        if constexpr (BACKWARD) emit<T, true, TERMS>(static_cast<T*>(p.zt) + at * (TERMS * kC * kC), zm);
        __syncthreads();
    }
}

template <typename T, int N, bool BACKWARD>
int launch_prep(const DeltaParams& p, hipStream_t stream) {
    hipLaunchKernelGGL((delta_prep_kernel<T, N, BACKWARD>), dim3((unsigned)(p.slots * p.G)), dim3(kThreads), 0, stream, p);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace delta
}  // namespace ssd
