// delta_walk_kernel: the states of the gated delta rule from chunk to chunk, and the outputs.
//
// For a chunk with entering state S, e^g and e^(gC - g) per token, and Z from delta_prep_kernel:
//     R = V - e^g (K S),  E = R + Z B R,  U = B E,  y = scale (e^g (Q S) + P U),  S' = e^gC S + K^T (e^(gC - g) U).
// The columns of S do not meet: a workgroup takes 32 of them (of one sequence and head) down the sequence.  Its four
// waves share the columns and split the rows: wave w has the chunk's tokens 16 w .. in R, E and y, and a quarter of
// S's rows in registers, fp32.  What all waves need of S, B R and U goes through LDS as operands of several terms; the other
// operands (rows of K and Q, and Z, P, K^T as delta_prep_kernel laid them out) come straight from memory, the next
// chunk's on their way while this one is worked on.  Three barriers a chunk.  Tile i of a lane m is column 2 m + i, so that a lane
// loads and stores pairs.
//
// SAVE (the backward pass's run of it): keeps the state before every chunk and after the last, e, and dy . y per token.
#pragma once

#include "ssd_delta_common.h"

namespace ssd {
namespace delta {

constexpr int CT = kCols / 16;  // column tiles of a walk's workgroup

// A wave's rows of a state [N][P]: tiles tile0 .. of 16 rows, NT of them.  (At N = 32 there are two tiles for four waves: the
// last two waves work on the last tile too, and do not store it.)
template <int N> struct StateRows {
    static constexpr int NT = (N / 16 + 3) / 4;
    static constexpr bool kAll = N / 16 >= kWaves;
    int tile0, m, g;
    bool own;
    __device__ __forceinline__ StateRows(int w, int lane) : m(lane % 16), g(lane / 16) {
        tile0 = kAll ? w * NT : min(w, N / 16 - 1);
        own = kAll || w < N / 16;
    }
    // to or from [N][P] at its column block
    __device__ __forceinline__ void load(f32x4 (&st)[NT][CT], const float* from, int P) const {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f32x2 x = from ? *reinterpret_cast<const f32x2*>(from + (16 * (tile0 + t) + 4 * g + e) * P + 2 * m) : f32x2{};
                st[t][0][e] = x[0];
                st[t][1][e] = x[1];
            }
    }
    __device__ __forceinline__ void store(const f32x4 (&st)[NT][CT], float* to, int P) const {
        if (!kAll && !own) return;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *reinterpret_cast<f32x2*>(to + (16 * (tile0 + t) + 4 * g + e) * P + 2 * m) = f32x2{st[t][0][e], st[t][1][e]};
    }
    // as operands [column][n] in LDS
    template <int TERMS, typename T> __device__ __forceinline__ void share(const f32x4 (&st)[NT][CT], T* sl, int row, int apart) const {
        if (!kAll && !own) return;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int c = 0; c < CT; ++c) put4<TERMS>(sl + (16 * c + m) * row + 16 * (tile0 + t) + 4 * g, apart, st[t][c]);
    }
};

template <typename T, int N, bool SAVE>
__global__ void __launch_bounds__(kThreads, N * sizeof(T) == 512 ? 1 : 2) delta_walk_kernel(DeltaParams p, int64_t units, int64_t per_xcd) {
    using M = Mat<T>;
    using Frag = typename M::Frag;
    constexpr int KN = N / M::kK, KC = kC / M::kK, TERMS = M::kTerms;
    constexpr int TY = SAVE || TERMS == 1 ? TERMS : 2;  // terms of what only y takes: a bf16 y of S and U in two, of P in one
    constexpr int TP = SAVE ? TERMS : 1;
    constexpr int NT = StateRows<N>::NT;
    constexpr int LS = N + M::kPad, LC = kC + M::kPad;
    constexpr int SA = kCols * LS, CA = kCols * LC;  // elements from one term to the next
    __shared__ __attribute__((aligned(16))) T sl[TERMS * SA];  // S   [column][n]
    __shared__ __attribute__((aligned(16))) T rl[TERMS * CA];  // B R [column][token]
    __shared__ __attribute__((aligned(16))) T dl[TERMS * CA];  // e^(gC - g) U
    __shared__ __attribute__((aligned(16))) T ul[TY * CA];     // U

    const int64_t unit = xcd_work_index(blockIdx.x, per_xcd, units);
    if (unit < 0) return;
    const int blocks = p.P / kCols, cb = (int)(unit % blocks), h = (int)(unit / blocks % p.H), grp = h / (p.H / p.G);
    const int64_t s = unit / blocks / p.H;
    const Span span = span_of(p, s);
    const int64_t slot0 = span.lo / kC + s, chunks = (span.len + kC - 1) / kC;
    const int lane = threadIdx.x % kWave, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), m = lane % 16, g = lane / 16;
    const int row0 = 16 * w + 4 * g;              // this lane's four tokens of a chunk
    const int ksz = (16 * w + 15) / M::kK + 1;    // steps with anything left of the diagonal
    const StateRows<N> rows(w, lane);
    const int64_t NP = (int64_t)N * p.P, HP = (int64_t)p.H * p.P;

    f32x4 st[NT][CT];
    rows.load(st, p.init ? p.init + (s * p.H + h) * NP + cb * kCols : nullptr, p.P);
    rows.template share<TERMS>(st, sl, LS, SA);

    Frag kf[KN], qf[KN], zf[KC][TERMS], pf[KC][TP], tf[NT][KC];
    f32x4 in, out, be;
    float all;
    T vv[4][CT], dyv[4][CT];
    const int64_t vcol = (int64_t)h * p.P + cb * kCols;
    const auto load_rows = [&](int64_t c) {
        const int64_t t0 = span.lo + c * kC, have = span.len - c * kC < kC ? span.len - c * kC : kC;
        const Rows<T> kr(static_cast<const T*>(p.k) + t0 * p.k_stride + grp * N, have, p.k_stride, N);
        const Rows<T> qr(static_cast<const T*>(p.q) + t0 * p.q_stride + grp * N, have, p.q_stride, N);
#pragma unroll
        for (int i = 0; i < KN; ++i) kf[i] = kr.frag(16 * w + m, i * M::kK + g * M::kE);
#pragma unroll
        for (int i = 0; i < KN; ++i) qf[i] = qr.frag(16 * w + m, i * M::kK + g * M::kE);
    };
    const auto load_values = [&](int64_t c) {
        const int64_t t0 = span.lo + c * kC, have = span.len - c * kC < kC ? span.len - c * kC : kC;
        const Rows<T> vr(static_cast<const T*>(p.v) + t0 * p.v_stride + vcol, have, p.v_stride, kCols);
        const float* gates = p.gates + ((slot0 + c) * p.H + h) * (kDeltaGates * kC);
        in = as_f32x4(ld16(gates + kGateIn * kC + row0));
        out = as_f32x4(ld16(gates + kGateOut * kC + row0));
        be = as_f32x4(ld16(gates + kGateBeta * kC + row0));
        all = gates[kGateIn * kC + kC - 1];
#pragma unroll
        for (int e = 0; e < 4; ++e) vr.load2(row0 + e, 2 * m, vv[e]);
    };
    const auto load_z = [&](int64_t c) {
        const T* z = static_cast<const T*>(p.z) + ((slot0 + c) * p.H + h) * (int64_t)(TERMS * kC * kC) + (w * KC * kWave + lane) * M::kE;
#pragma unroll
        for (int i = 0; i < KC; ++i)
#pragma unroll
            for (int u = 0; u < TERMS; ++u) zf[i][u] = frag(z + u * (kC * kC) + min(i, ksz - 1) * (kWave * M::kE));
    };
    const auto load_rest = [&](int64_t c) {
        const T* sc = static_cast<const T*>(p.scores) + ((slot0 + c) * p.H + h) * (int64_t)(TP * kC * kC) + (w * KC * kWave + lane) * M::kE;
        const T* kt = static_cast<const T*>(p.kt) + ((slot0 + c) * p.G + grp) * (int64_t)(N * kC) + (rows.tile0 * KC * kWave + lane) * M::kE;
#pragma unroll
        for (int i = 0; i < KC; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t) tf[t][i] = frag(kt + (t * KC + i) * (kWave * M::kE));
#pragma unroll
        for (int i = 0; i < KC; ++i)
#pragma unroll
            for (int u = 0; u < TP; ++u) pf[i][u] = frag(sc + u * (kC * kC) + min(i, ksz - 1) * (kWave * M::kE));
        if constexpr (SAVE) {
            const int64_t t0 = span.lo + c * kC, have = span.len - c * kC < kC ? span.len - c * kC : kC;
            const Rows<T> yr(static_cast<const T*>(p.dy) + t0 * HP + vcol, have, HP, kCols);
#pragma unroll
            for (int e = 0; e < 4; ++e) yr.load2(row0 + e, 2 * m, dyv[e]);
        }
    };
    if (chunks > 0) {
        load_rows(0);
        load_z(0);
        load_values(0);
        load_rest(0);
    }
    for (int64_t c = 0; c < chunks; ++c) {
        const int64_t next = c + 1 < chunks ? c + 1 : c;
        if constexpr (SAVE) rows.store(st, p.states + ((slot0 + c + s) * p.H + h) * NP + cb * kCols, p.P);
        lds_barrier();  // S is there
        f32x4 r[CT], y[CT];
#pragma unroll
        for (int i = 0; i < CT; ++i) {
            const T* b = sl + (16 * i + m) * LS + g * M::kE;
            f32x4 a{};
            y[i] = f32x4{};
#pragma unroll
            for (int t = 0; t < KN; ++t) a = mma_terms<T, 1, TERMS>(&kf[t], b + t * M::kK, SA, a);
#pragma unroll
            for (int t = 0; t < KN; ++t) y[i] = mma_terms<T, 1, TY>(&qf[t], b + t * M::kK, SA, y[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) r[i][e] = to_f32(vv[e][i]) - in[e] * a[e];
            put4<TERMS>(rl + (16 * i + m) * LC + M::place_of(w, g), CA, be * r[i]);
        }
        load_rows(next);
        lds_barrier();  // B R is there, S is free
        f32x4 u[CT];
#pragma unroll
        for (int i = 0; i < CT; ++i) {
#pragma unroll
            for (int t = 0; t < KC; ++t)
                if (t < ksz) r[i] = mma_terms<T, TERMS, TERMS>(zf[t], rl + (16 * i + m) * LC + t * M::kK + g * M::kE, CA, r[i]);
            u[i] = be * r[i];
            put4<TERMS>(dl + (16 * i + m) * LC + M::place_of(w, g), CA, out * u[i]);
            put4<TY>(ul + (16 * i + m) * LC + M::place_of(w, g), CA, u[i]);
            y[i] *= in;
        }
        const float now = all;
        load_z(next);
        load_values(next);
        lds_barrier();  // U is there, B R is free
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < CT; ++i) {
                st[t][i] *= now;
#pragma unroll
                for (int k = 0; k < KC; ++k)
                    st[t][i] = mma_terms<T, 1, TERMS>(&tf[t][k], dl + (16 * i + m) * LC + k * M::kK + g * M::kE, CA, st[t][i]);
            }
        rows.template share<TERMS>(st, sl, LS, SA);
#pragma unroll
        for (int i = 0; i < CT; ++i) {
#pragma unroll
            for (int t = 0; t < KC; ++t)
                if (t < ksz) y[i] = mma_terms<T, TP, TY>(pf[t], ul + (16 * i + m) * LC + t * M::kK + g * M::kE, CA, y[i]);
            y[i] *= p.scale;
        }
        const int64_t t0 = span.lo + c * kC, have = span.len - c * kC < kC ? span.len - c * kC : kC;
        if constexpr (SAVE) {
            const Rows<float> er(p.wrong + t0 * HP + vcol, have, HP, kCols);
            f32x4 dot;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                er.store2(row0 + e, 2 * m, r[0][e], r[1][e]);
                dot[e] = sum16(y[0][e] * to_f32(dyv[e][0]) + y[1][e] * to_f32(dyv[e][1]));
            }
            if (m == 0) st16(p.dot_y + (((slot0 + c) * p.H + h) * blocks + cb) * kC + row0, __builtin_bit_cast(uint4, dot));
        } else {
            const Rows<T> yr(static_cast<T*>(p.y) + t0 * HP + vcol, have, HP, kCols);
#pragma unroll
            for (int e = 0; e < 4; ++e) yr.store2(row0 + e, 2 * m, y[0][e], y[1][e]);
        }
        load_rest(next);
    }
    if constexpr (SAVE) rows.store(st, p.states + ((slot0 + chunks + s) * p.H + h) * NP + cb * kCols, p.P);
    else if (p.final_state) rows.store(st, p.final_state + (s * p.H + h) * NP + cb * kCols, p.P);
}

template <typename T, int N, bool SAVE>
int launch_walk(const DeltaParams& p, hipStream_t stream) {
    const int64_t units = p.nseq * p.H * (p.P / kCols), per = (units + 7) / 8;
    hipLaunchKernelGGL((delta_walk_kernel<T, N, SAVE>), dim3((unsigned)(8 * per)), dim3(kThreads), 0, stream, p, units, per);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace delta
}  // namespace ssd
