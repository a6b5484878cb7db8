// delta_walk_kernel: the states of the gated delta rule from chunk to chunk, and the outputs.
//
// For a chunk with entering state S, e^g and e^(gC - g) per token, and Z from delta_prep_kernel:
//     R = V - e^g (K S),  E = R + Z B R,  U = B E,  y = scale (e^g (Q S) + P U),  S' = e^gC S + K^T (e^(gC - g) U).
// The columns of S do not meet: a workgroup takes 16 or 32 of them (of one sequence and head) down the sequence.  Its four
// waves share the columns and split the rows: wave w has the chunk's tokens 16 w .. in R, E and y, and a quarter of
// S's rows in registers, fp32.  What all waves need of S, B R and U goes through LDS as operands of several terms; the other
// operands (K, Q, Z, P as delta_prep_kernel laid them out) come straight from memory, the next
// chunk's on their way while this one is worked on.  Three barriers a chunk (four where U has the place of S).  Where there are two tiles of
// 16 columns, tile i of lane m is column 2 m + i, so that a lane loads and stores pairs.
//
// Bound by the chain of a chunk: three barriers, two products of each kind after another and the splitting into
// terms in between, on one or two waves a SIMD, with the operands' way through the CU's L1 next (77 KB a chunk at 128 keys).  16384
// tokens, 32/16 heads of 128 by 128, bf16: 256 chunks in 551 us, 2.15 us each (with its loads left out 1.45: the loads are
// half hidden); 8 x 2048 tokens, 24 heads of 128 by 64, two workgroups on every other CU: 167 us, 494 MB read and 54 written (3.3 TB/s), and
// 255 us with SAVE, 568 and 311 MB (3.4 TB/s; 300 us with one workgroup a CU).  There the bytes, most of them operands of several terms
// made for the walks, are two thirds of the time at the rate of a copy.
//
// SAVE (the backward pass's run of it): keeps the state before every chunk and after the last, e, and dy . y per token.
#pragma once

#include "ssd_delta_common.h"

namespace ssd {
namespace delta {

// A wave's rows of a state [N][P]: tiles tile0 .. of 16 rows, NT of them.  (At N = 32 there are two tiles for four waves: the
// last two waves work on the last tile too, and do not store it.)
template <int N, int CT> struct StateRows {
    static constexpr int NT = (N / 16 + 3) / 4;
    static constexpr bool kAll = N / 16 >= kWaves;
    int tile0, m, g;
    bool own;
    __device__ __forceinline__ StateRows(int w, int lane) : m(lane % 16), g(lane / 16) {
        tile0 = kAll ? w * NT : min(w, N / 16 - 1);
        own = kAll || w < N / 16;
    }
    // to or from [N][P] at its column block
    __device__ __forceinline__ uint32_t at(int t, int e, int P) const { return (uint32_t)(((16 * (tile0 + t) + 4 * g + e) * P + CT * m) * 4); }
    __device__ __forceinline__ void load(f32x4 (&st)[NT][CT], const float* from, int P) const {
        const Block b(from);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x[CT] = {};
                if (from) b.load<CT>(at(t, e, P), x);
#pragma unroll
                for (int i = 0; i < CT; ++i) st[t][i][e] = x[i];
            }
    }
    template <typename T> __device__ __forceinline__ void store(const f32x4 (&st)[NT][CT], T* to, int P) const {
        if (!kAll && !own) return;
        const Block b(to);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x[CT];
#pragma unroll
                for (int i = 0; i < CT; ++i) x[i] = st[t][i][e];
                b.store<CT, T>(at(t, e, P) / (4 / sizeof(T)), x);
            }
    }
    // what their rounding to bf16 leaves, rounded to bf16
    __device__ __forceinline__ void store_rest(const f32x4 (&st)[NT][CT], __bf16* to, int P) const {
        f32x4 rest[NT][CT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < CT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) rest[t][i][e] = st[t][i][e] - (float)(__bf16)st[t][i][e];
        store(rest, to, P);
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

// Whether U has the place of S between its reading and its next writing, for one barrier more: where two workgroups would not
// fit a CU's LDS otherwise.  Z and P are then loaded one after the other, in the chunk that takes them, to stay within 256 registers.
// 8 x 2048 tokens, 24 heads of 128 by 64, bf16 (384 workgroups): 300 us with a CU each, 253 so.
template <typename T, int N, int CT, bool SAVE> constexpr bool walk_shares() { return SAVE && CT == 2 && N == 128 && sizeof(T) == 2; }

template <typename T, int N, int CT, bool SAVE>
__global__ void __launch_bounds__(kThreads, CT == 2 && N * sizeof(T) == 512 ? 1 : 2) delta_walk_kernel(DeltaParams p, int64_t units, int64_t per_xcd) {
    using M = Mat<T>;
    using Frag = typename M::Frag;
    constexpr int KN = N / M::kK, KC = kC / M::kK, TERMS = M::kTerms;
    constexpr int TY = terms_of_y<T>(SAVE);  // of what only y takes
    constexpr int NT = StateRows<N, CT>::NT, kCols = 16 * CT;
    constexpr int LS = N + M::kPad, LC = kC + M::kPad;
    constexpr int SA = kCols * LS, CA = kCols * LC;  // elements from one term to the next
    constexpr bool SHARED = walk_shares<T, N, CT, SAVE>();
    extern __shared__ __attribute__((aligned(16))) char walk_lds[];
    T* const sl = reinterpret_cast<T*>(walk_lds);  // S   [column][n]
    T* const rl = sl + TERMS * SA;                 // B R [column][token]
    T* const dl = rl + TERMS * CA;                 // e^(gC - g) U
    T* const ul = SHARED ? sl : dl + TERMS * CA;   // U
    T* const kl = dl + (TERMS + (SHARED ? 0 : TY)) * CA;  // K   [token][n]

    const int64_t unit = xcd_work_index(blockIdx.x, per_xcd, units);
    if (unit < 0) return;
    const int blocks = p.P / kCols, cb = (int)(unit % blocks), h = (int)(unit / blocks % p.H), grp = h / (p.H / p.G);
    const int64_t s = unit / blocks / p.H;
    const Span span = span_of(p, s);
    const int64_t slot0 = span.lo / kC + s, chunks = (span.len + kC - 1) / kC;
    const int lane = threadIdx.x % kWave, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), m = lane % 16, g = lane / 16;
    const int row0 = 16 * w + 4 * g;              // this lane's four tokens of a chunk
    const int ksz = (16 * w + 15) / M::kK + 1;    // steps with anything left of the diagonal
    const StateRows<N, CT> rows(w, lane);
    const int64_t NP = (int64_t)N * p.P, HP = (int64_t)p.H * p.P;

    f32x4 st[NT][CT];
    rows.load(st, p.init ? p.init + (s * p.H + h) * NP + cb * kCols : nullptr, p.P);
    rows.template share<TERMS>(st, sl, LS, SA);

    const T *const at_s = sl + m * LS + g * M::kE, *const at_r = rl + m * LC + g * M::kE, *const at_d = dl + m * LC + g * M::kE,
            *const at_u = ul + m * LC + g * M::kE;
    Frag kf[KN], qf[KN], zf[KC][TERMS], pf[KC][TY];
    f32x4 in, out, be, in1, out1, be1;  // the latter of the next chunk: what is used first in a chunk is loaded a whole one before
    float all, all1;
    T vv[4][CT], dyv[4][CT];
    constexpr uint32_t kStep = kWave * 16;  // bytes of an operand of all lanes
    const int64_t vcol = (int64_t)h * p.P + cb * kCols;
    Chunks vc(static_cast<const T*>(p.v) + span.lo * p.v_stride + vcol, span.len, p.v_stride, kCols);
    Chunks yc(static_cast<const T*>(SAVE ? p.dy : p.y) + span.lo * HP + vcol, span.len, HP, kCols);  // y; SAVE: dy
    Chunks ec(p.wrong + span.lo * HP + vcol, span.len, HP, kCols);
    const int64_t row_at = (slot0 * p.G + grp) * (int64_t)(N * kC * sizeof(T));
    const char *kc = static_cast<const char*>(p.kr) + row_at + w * KN * kStep, *qc = static_cast<const char*>(p.qr) + row_at + w * KN * kStep;
    const char* zc = static_cast<const char*>(p.z) + (slot0 * p.H + h) * (int64_t)(TERMS * kC * kC * sizeof(T)) + w * KC * kStep;
    const char* pc = static_cast<const char*>(p.scores) + (slot0 * p.H + h) * (int64_t)(TY * kC * kC * sizeof(T)) + w * KC * kStep;
    const float* gc = p.gates + (slot0 * p.H + h) * (kDeltaGates * kC);
    const uint32_t own = lane * 16, four = row0 * 4;
    uint32_t vat[4], yat[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        vat[e] = (uint32_t)(((row0 + e) * p.v_stride + CT * m) * sizeof(T));
        yat[e] = (uint32_t)(((row0 + e) * HP + CT * m) * sizeof(T));
    }
    // loads of the chunk `on` chunks (1, or 0 behind the last one) from the one loaded before, which is the sequence's last or not
    const auto load_rows = [&](int64_t on) {
        kc += on * (p.G * (int64_t)(N * kC * sizeof(T)));
        qc += on * (p.G * (int64_t)(N * kC * sizeof(T)));
        const Block kr(kc), qr(qc);
#pragma unroll
        for (int i = 0; i < KN; ++i) kf[i] = kr.frag<T>(own, i * kStep);
#pragma unroll
        for (int i = 0; i < KN; ++i) qf[i] = qr.frag<T>(own, i * kStep);
    };
    const auto load_gates = [&](int64_t on) {
        gc += on * (p.H * (kDeltaGates * kC));
        const Block gr(gc);
        in1 = as_f32x4(gr.load16(four, kGateIn * kC * 4));
        out1 = as_f32x4(gr.load16(four, kGateOut * kC * 4));
        be1 = as_f32x4(gr.load16(four, kGateBeta * kC * 4));
        all1 = gc[kGateIn * kC + kC - 1];
    };
    const auto load_values = [&](int64_t on, bool last) {
        vc.base += on * vc.step;
        const Block vr = vc.block(last);
#pragma unroll
        for (int e = 0; e < 4; ++e) vr.load<CT>(vat[e], vv[e]);
    };
    const auto load_z = [&](int64_t on) {
        zc += on * (p.H * (int64_t)(TERMS * kC * kC * sizeof(T)));
        const Block z(zc);
#pragma unroll
        for (int i = 0; i < KC; ++i)
#pragma unroll
            for (int u = 0; u < TERMS; ++u) zf[i][u] = z.frag<T>(i < ksz ? own + i * kStep : own, u * (kC * kC * sizeof(T)));
    };
    const auto load_rest = [&](int64_t on, bool last) {
        pc += on * (p.H * (int64_t)(TY * kC * kC * sizeof(T)));
        if constexpr (SAVE) yc.base += on * yc.step;
        const Block sc(pc);
#pragma unroll
        for (int i = 0; i < KC; ++i)
#pragma unroll
            for (int u = 0; u < TY; ++u) pf[i][u] = sc.frag<T>(i < ksz ? own + i * kStep : own, u * (kC * kC * sizeof(T)));
        if constexpr (SAVE) {
            const Block yr = yc.block(last);
#pragma unroll
            for (int e = 0; e < 4; ++e) yr.load<CT>(yat[e], dyv[e]);
        }
    };
    if (chunks > 0) {
        load_rows(0);
        load_gates(0);
        load_z(0);
        load_values(0, chunks == 1);
        if constexpr (!SHARED) load_rest(0, chunks == 1);
    }
    float* keep = SAVE ? p.states + ((slot0 + s) * p.H + h) * NP + cb * kCols : nullptr;
    for (int64_t c = 0; c < chunks; ++c) {
        const int64_t on = c + 1 < chunks;
        const bool last = c + 2 >= chunks;
        if constexpr (SAVE) {
            rows.store(st, keep, p.P);
            keep += p.H * NP;
        }
        in = in1;
        out = out1;
        be = be1;
        all = all1;
        load_gates(on);
        lds_barrier();  // S is there
        f32x4 a[CT] = {}, y[CT] = {}, r[CT];
        {
            Operands<T, CT, TERMS> b[2];
            b[0].read(at_s, 0, 16 * LS, SA);
#pragma unroll
            for (int t = 0; t < KN; ++t) {
                if (t + 1 < KN) b[(t + 1) % 2].read(at_s, t + 1, 16 * LS, SA);
                __builtin_amdgcn_sched_barrier(0);
                b[t % 2].template add<1>(a, &kf[t]);
                Operands<T, CT, TY> by;
#pragma unroll
                for (int i = 0; i < CT; ++i)
#pragma unroll
                    for (int u = 0; u < TY; ++u) by.f[i][u] = b[t % 2].f[i][u];
                by.template add<1>(y, &qf[t]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int i = 0; i < CT; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) r[i][e] = to_f32(vv[e][i]) - in[e] * a[i][e];
            put4<TERMS>(rl + (16 * i + m) * LC + M::place_of(w, g), CA, be * r[i]);
        }
        // (K's columns are the state's other operand: by way of LDS)
#pragma unroll
        for (int t = 0; t < KN; ++t) st16(kl + (16 * w + m) * LS + t * M::kK + g * M::kE, __builtin_bit_cast(uint4, kf[t]));
        load_rows(on);
        load_values(on, last);
        lds_barrier();  // B R is there, S is free
        f32x4 u[CT];
        {
            Operands<T, CT, TERMS> b[KC];
#pragma unroll
            for (int t = 0; t < KC; ++t)
                if (t < ksz) b[t].read(at_r, t, 16 * LC, CA);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < KC; ++t)
                if (t < ksz) b[t].template add<TERMS>(r, zf[t]);
        }
#pragma unroll
        for (int i = 0; i < CT; ++i) {
            u[i] = be * r[i];
            put4<TERMS>(dl + (16 * i + m) * LC + M::place_of(w, g), CA, out * u[i]);
            put4<TY>(ul + (16 * i + m) * LC + M::place_of(w, g), CA, u[i]);
            y[i] *= in;
        }
        // (two workgroups have registers for one of Z and P at a time)
        if constexpr (SHARED) load_rest(c > 0, !on);
        else load_z(on);
        lds_barrier();  // U is there, B R is free
        {
            Operands<T, CT, TERMS> b[KC];
            Frag tf[NT][KC];
#pragma unroll
            for (int k = 0; k < KC; ++k) {
                b[k].read(at_d, k, 16 * LC, CA);
#pragma unroll
                for (int t = 0; t < NT; ++t) tf[t][k] = columns_of(kl, LS, 16 * (rows.tile0 + t), k, m, g);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < CT; ++i) st[t][i] *= all;
#pragma unroll
            for (int k = 0; k < KC; ++k)
#pragma unroll
                for (int t = 0; t < NT; ++t) b[k].template add<1>(st[t], &tf[t][k]);
        }
        Operands<T, CT, TY> b[KC];
#pragma unroll
        for (int t = 0; t < KC; ++t) b[t].read(at_u, t, 16 * LC, CA);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (SHARED) lds_barrier();  // U is free
        rows.template share<TERMS>(st, sl, LS, SA);
#pragma unroll
        for (int t = 0; t < KC; ++t)
            if (t < ksz) b[t].template add<TY>(y, pf[t]);
#pragma unroll
        for (int i = 0; i < CT; ++i) y[i] *= p.scale;
        if constexpr (SAVE) {
            const Block er = ec.block(!on);
            f32x4 dot;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x[CT], sum = 0.f;
#pragma unroll
                for (int i = 0; i < CT; ++i) {
                    x[i] = r[i][e];
                    sum += y[i][e] * to_f32(dyv[e][i]);
                }
                er.store<CT, float>(yat[e] * (4 / sizeof(T)), x);
                dot[e] = sum16(sum);
            }
            ec.base += ec.step;
            if (m == 0) st16(p.dot_y + (((slot0 + c) * p.H + h) * blocks + cb) * kC + row0, __builtin_bit_cast(uint4, dot));
        } else {
            const Block yr = yc.block(!on);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x[CT];
#pragma unroll
                for (int i = 0; i < CT; ++i) x[i] = y[i][e];
                yr.store<CT, T>(yat[e], x);
            }
            yc.base += yc.step;
        }
        if constexpr (SHARED) load_z(on);
        else load_rest(on, last);
    }
    if constexpr (SAVE) rows.store(st, keep, p.P);
    else if (p.final_state) rows.store(st, p.final_state + (s * p.H + h) * NP + cb * kCols, p.P);
}

template <typename T, int N, int CT, bool SAVE>
int launch_walk(const DeltaParams& p, hipStream_t stream) {
    using M = Mat<T>;
    const int64_t units = p.nseq * p.H * (p.P / (16 * CT)), per = (units + 7) / 8;
    constexpr int TY = terms_of_y<T>(SAVE), LS = N + M::kPad, LC = kC + M::kPad;
    constexpr int lds = (16 * CT * (M::kTerms * LS + (2 * M::kTerms + (walk_shares<T, N, CT, SAVE>() ? 0 : TY)) * LC) + kC * LS) * (int)sizeof(T);
    const auto kernel = &delta_walk_kernel<T, N, CT, SAVE>;
    if (hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, lds) != hipSuccess) return -1;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(8 * per)), dim3(kThreads), lds, stream, p, units, per);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}
template <typename T, int N, bool SAVE> int launch_walk(const DeltaParams& p, hipStream_t stream) {
    return p.cols == 16 ? launch_walk<T, N, 1, SAVE>(p, stream) : launch_walk<T, N, 2, SAVE>(p, stream);
}

}  // namespace delta
}  // namespace ssd
