// The backward pass of the gated delta rule, gfx950.  With the notation of ssd_delta_walk.h, x the gradient that reaches
// U = B E, and dS' the gradient of the state after a chunk:
//     dU = scale P^T dY + e^(gC - g) (K dS'),  x = dU + Z^T B dU,  dE = B x = dV,
//     dS = e^gC dS' + scale Q^T (e^g dY) - K^T (e^g dE),
//     dbeta_i = x_i . e_i,
//     dlog a_t = F_{t-1} = F_t + dy_t . y_t - dv_t . v_t,  F_t = <gradient of S_t, S_t>
// (a step's decay multiplies all of the state before it; the sums of the other gradients telescope).  F is known on both sides
// of a chunk, as <dS', S'> and <dS, S>, and what the sum from the one misses the other by is rounding: it is spread over
// the chunk's tokens evenly, so that the error of each is that of the shorter way (fp32, 901 tokens in documents of odd lengths:
// 6e-7 of dlog a, against 1.1e-6 of the one sum).  And
//     dq_i = scale (e^g_i S dy_i + sum_{j<=i} D_ij (dy_i.u_j) k_j)
//     dk_i = scale sum_{l>=i} D_li (dy_l.u_i) q_l - sum_{l>i} D_li (de_l.u_i) k_l - sum_{j<i} D_ij (de_i.u_j) k_j
//            + e^(gC - g_i) dS' u_i - e^g_i S de_i.
// Four launches: delta_prep_kernel and delta_walk_kernel again (which keep the states before the chunks, e and dy . y),
// delta_back_kernel down the chunks from the last one, delta_grad_kernel for dq, dk and the sums, all chunks at once.
#include <type_traits>

#include "ssd_delta_prep.h"
#include "ssd_delta_walk.h"

namespace ssd {
namespace delta {
namespace {

// The gradient of the state, from chunk to chunk towards the first: as delta_walk_kernel, 16 or 32 columns a workgroup, the
// rows split over its waves, every product of fp32 values on operands of all terms.
// Bound as there by a chunk's chain and by bytes: 8 x 2048 tokens, 24 heads of 128 by 64, bf16, 309 us, 856 MB read and 317 written (3.8 TB/s;
// 278 us without the second terms of dS' and dV that it stores for dq and dk).
//
// Whether a workgroup of 32 columns keeps to half of a CU, 256 registers a lane and 80 KB: it then loads Z, Q, the values
// and the state in the chunk that takes them, under the products before, and not a chunk ahead.  With a CU each and so, us, 64 values a head:
//     workgroups (sequences)     256 (4 x 2048)    384 (8 x 2048)    1024 (16 x 1024)
//     bf16, keys of 32           189 151           264 216           285 237
//                   64           165 160           296 245           329 271
//                  128           189 186           364 305           (256: 128 values)
//     fp32, keys of 32           174 167           249 232           284 265
//                   64           189 176           348 266           381 308
// (fp32 operands of 128 keys do not fit a half.)
template <typename T, int N, int CT> constexpr bool back_lean() { return CT == 2 && N * sizeof(T) <= 256; }
// Whether a workgroup may take all of a CU's registers: for fp32 keys of 128, which need more than half and have the CU for themselves
// anyway, with 16 columns as 256 workgroups at most, with 32 by their LDS (four sequences of 2048 tokens, 16 heads of 128 by 64: 177 us; within
// half, 16 registers spilled, 228).
template <typename T, int N> constexpr bool back_alone() { return N * sizeof(T) > 256; }

template <typename T, int N, int CT>
__global__ void __launch_bounds__(kThreads, (back_alone<T, N>() ? 1 : 2)) delta_back_kernel(DeltaParams p, int64_t units, int64_t per_xcd) {
    using M = Mat<T>;
    using Frag = typename M::Frag;
    constexpr int KN = N / M::kK, KC = kC / M::kK, TERMS = M::kTerms, NT = StateRows<N, CT>::NT, kCols = 16 * CT;
    constexpr int LS = N + M::kPad, LC = kC + M::kPad, SA = kCols * LS, CA = kCols * LC;
    constexpr bool LEAN = back_lean<T, N, CT>();
    // dS' [column][n], and in its place, between its reading and its next writing, K and Q [token][n]; dY [column][token]; of
    // all terms: scale e^g dY, B dU, -e^g dE
    extern __shared__ __attribute__((aligned(16))) char back_lds[];
    T* const sl = reinterpret_cast<T*>(back_lds);
    T *const kl = sl, *const ql = kl + kC * LS;
    T* const yl = sl + (TERMS * SA > 2 * kC * LS ? TERMS * SA : 2 * kC * LS);
    T* const wl = yl + CA;
    T* const rl = wl + TERMS * CA;
    T* const dl = rl + TERMS * CA;

    const int64_t unit = xcd_work_index(blockIdx.x, per_xcd, units);
    if (unit < 0) return;
    const int blocks = p.P / kCols, cb = (int)(unit % blocks), h = (int)(unit / blocks % p.H), grp = h / (p.H / p.G);
    const int64_t s = unit / blocks / p.H;
    const Span span = span_of(p, s);
    const int64_t slot0 = span.lo / kC + s, chunks = (span.len + kC - 1) / kC;
    const int lane = threadIdx.x % kWave, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), m = lane % 16, g = lane / 16;
    const int row0 = 16 * w + 4 * g, ks0 = 16 * w / M::kK;  // (steps before ks0 are left of the diagonal: zero)
    const StateRows<N, CT> rows(w, lane);
    const int64_t NP = (int64_t)N * p.P, HP = (int64_t)p.H * p.P, vcol = (int64_t)h * p.P + cb * kCols;

    f32x4 st[NT][CT];
    rows.load(st, p.dfinal ? p.dfinal + (s * p.H + h) * NP + cb * kCols : nullptr, p.P);
    rows.template share<TERMS>(st, sl, LS, SA);

    const T *const at_s = sl + m * LS + g * M::kE, *const at_y = yl + m * LC + g * M::kE, *const at_w = wl + m * LC + g * M::kE,
            *const at_r = rl + m * LC + g * M::kE, *const at_d = dl + m * LC + g * M::kE;
    Frag kf[KN], qf[KN], zf[KC][TERMS], pf[KC][TERMS];
    f32x4 in, out, be, after[NT][CT];
    float all;
    T vv[4][CT], yv[4][CT];
    float ee[4][CT];
    constexpr uint32_t kStep = kWave * 16;  // bytes of an operand of all lanes
    const int64_t end = chunks - 1, kept = chunks > 0 ? end : 0;  // (the chunks are taken from the last one on)
    const auto to_last = [&](Chunks x) {
        x.base += kept * x.step;
        return x;
    };
    Chunks vc = to_last(Chunks(static_cast<const T*>(p.v) + span.lo * p.v_stride + vcol, span.len, p.v_stride, kCols));
    Chunks yc = to_last(Chunks(static_cast<const T*>(p.dy) + span.lo * HP + vcol, span.len, HP, kCols));
    Chunks oc = to_last(Chunks(static_cast<const T*>(p.dv) + span.lo * HP + vcol, span.len, HP, kCols));
    Chunks lc = to_last(Chunks(static_cast<const T*>(p.dv_rest) + span.lo * HP + vcol, span.len, HP, kCols));  // (bf16)
    Chunks ec = to_last(Chunks(p.wrong + span.lo * HP + vcol, span.len, HP, kCols));
    constexpr int64_t kMat = TERMS * kC * kC * sizeof(T), kCol = N * kC * sizeof(T), kGate = kDeltaGates * kC;
    const int64_t slot = slot0 + kept;
    const char* zc = static_cast<const char*>(p.zt) + (slot * p.H + h) * kMat + w * KC * kStep;
    const char* pc = static_cast<const char*>(p.scores_t) + (slot * p.H + h) * kMat + w * KC * kStep;
    const int64_t row_at = (slot * p.G + grp) * kCol + w * KN * kStep;
    const char *kc = static_cast<const char*>(p.kr) + row_at, *qc = static_cast<const char*>(p.qr) + row_at;
    const float* gc = p.gates + (slot * p.H + h) * kGate;
    const float* sc = p.states + ((slot + 1 + s) * p.H + h) * NP + cb * kCols;
    T* dc = static_cast<T*>(p.dstates) + (slot * p.H + h) * NP + cb * kCols;
    const int64_t rest_of = static_cast<T*>(p.dstates_rest) - static_cast<T*>(p.dstates);  // (bf16)
    const uint32_t own = lane * 16, four = row0 * 4;
    uint32_t vat[4], yat[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        vat[e] = (uint32_t)(((row0 + e) * p.v_stride + CT * m) * sizeof(T));
        yat[e] = (uint32_t)(((row0 + e) * HP + CT * m) * sizeof(T));
    }
    // loads of the chunk `back` chunks (1, or 0 before the first one) from the one loaded before, which is the last or not
    const auto load_rows = [&](int64_t back) {
        kc -= back * (p.G * kCol);
        pc -= back * (p.H * kMat);
        const Block kr(kc), s(pc);
#pragma unroll
        for (int i = 0; i < KN; ++i) kf[i] = kr.frag<T>(own, i * kStep);
#pragma unroll
        for (int i = 0; i < KC; ++i)
#pragma unroll
            for (int u = 0; u < TERMS; ++u) pf[i][u] = s.frag<T>(i < ks0 ? own + ks0 * kStep : own + i * kStep, u * (kC * kC * sizeof(T)));
    };
    const auto load_q = [&](int64_t back) {
        qc -= back * (p.G * kCol);
        const Block qr(qc);
#pragma unroll
        for (int i = 0; i < KN; ++i) qf[i] = qr.frag<T>(own, i * kStep);
    };
    const auto load_z = [&](int64_t back) {
        zc -= back * (p.H * kMat);
        const Block z(zc);
#pragma unroll
        for (int i = 0; i < KC; ++i)
#pragma unroll
            for (int u = 0; u < TERMS; ++u) zf[i][u] = z.frag<T>(i < ks0 ? own + ks0 * kStep : own + i * kStep, u * (kC * kC * sizeof(T)));
    };
    const auto load_values = [&](int64_t back, bool last) {
        vc.base -= back * vc.step;
        ec.base -= back * ec.step;
        const Block vr = vc.block(last), er = ec.block(last);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            vr.load<CT>(vat[e], vv[e]);
            er.load<CT>(yat[e] * (4 / sizeof(T)), ee[e]);
        }
    };
    const auto load_gates = [&](int64_t back) {
        gc -= back * (p.H * kGate);
        const Block gr(gc);
        in = as_f32x4(gr.load16(four, kGateIn * kC * 4));
        out = as_f32x4(gr.load16(four, kGateOut * kC * 4));
        be = as_f32x4(gr.load16(four, kGateBeta * kC * 4));
        all = gc[kGateIn * kC + kC - 1];
    };
    const auto load_after = [&](int64_t back) {
        sc -= back * (p.H * NP);
        rows.load(after, sc, p.P);
    };
    const auto load_dy = [&](int64_t back, bool last) {
        yc.base -= back * yc.step;
        const Block yr = yc.block(last);
#pragma unroll
        for (int e = 0; e < 4; ++e) yr.load<CT>(yat[e], yv[e]);
    };
    const auto share_dy = [&] {
#pragma unroll
        for (int i = 0; i < CT; ++i) {
            const f32x4 x = {to_f32(yv[0][i]), to_f32(yv[1][i]), to_f32(yv[2][i]), to_f32(yv[3][i])};
            put4<1>(yl + (16 * i + m) * LC + M::place_of(w, g), 0, x);
        }
    };
    // this wave's share of <gradient of the state, the state>
    const auto state_dot = [&] {
        float dot = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < CT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) dot += st[t][i][e] * after[t][i][e];
        if (!StateRows<N, CT>::kAll && !rows.own) dot = 0.f;
        dot = sum16(dot);
        dot += __shfl_xor(dot, 16, kWave);
        return dot + __shfl_xor(dot, 32, kWave);
    };
    if (chunks > 0) {
        load_dy(0, true);
        load_rows(0);
        if constexpr (!LEAN) {
            load_q(0);
            load_z(0);
            load_values(0, true);
            load_after(0);
        }
        load_gates(0);
        share_dy();
        load_dy(chunks > 1, chunks == 1);
    }
    for (int64_t c = chunks - 1; c >= 0; --c) {
        const int64_t back = c > 0, at = (slot0 + c) * p.H + h;
        const bool last = c == end && c == 0;  // of the chunk to load: the present one again, before the first
        rows.store(st, dc, p.P);
        if constexpr (TERMS > 1) rows.store_rest(st, dc + rest_of, p.P);
        dc -= p.H * NP;
        lds_barrier();  // dS' and dY are there
        f32x4 a[CT] = {}, d[CT] = {}, x[CT];
        {
            Operands<T, CT, 1> y[KC];
            Operands<T, CT, TERMS> b[2];
            b[0].read(at_s, 0, 16 * LS, SA);
#pragma unroll
            for (int t = 0; t < KC; ++t)
                if (t >= ks0) y[t].read(at_y, t, 16 * LC, 0);
#pragma unroll
            for (int t = 0; t < KN; ++t) {
                if (t + 1 < KN) b[(t + 1) % 2].read(at_s, t + 1, 16 * LS, SA);
                __builtin_amdgcn_sched_barrier(0);
                b[t % 2].template add<1>(a, &kf[t]);
            }
#pragma unroll
            for (int t = 0; t < KC; ++t)
                if (t >= ks0) y[t].template add<TERMS>(d, pf[t]);
        }
        if constexpr (LEAN) {
            load_z(c < end);
            load_q(c < end);
            load_values(c < end, c == end);
            load_after(c < end);
        }
#pragma unroll
        for (int i = 0; i < CT; ++i) {
            x[i] = p.scale * d[i] + out * a[i];
            put4<TERMS>(rl + (16 * i + m) * LC + M::place_of(w, g), CA, be * x[i]);
        }
        lds_barrier();  // B dU is there, dS' and dY are free
        // (K's and Q's columns are the state's other operands: by way of LDS)
#pragma unroll
        for (int t = 0; t < KN; ++t) {
            st16(kl + (16 * w + m) * LS + t * M::kK + g * M::kE, __builtin_bit_cast(uint4, kf[t]));
            st16(ql + (16 * w + m) * LS + t * M::kK + g * M::kE, __builtin_bit_cast(uint4, qf[t]));
        }
        if constexpr (!LEAN) {
            load_rows(back);
            load_q(back);
        }
        f32x4 dv{}, db{};
        const Block dr = oc.block(c == end);
        oc.base -= oc.step;
        const Block lr = lc.block(c == end);
        lc.base -= lc.step;
        f32x4 de[CT];
        {
            Operands<T, CT, TERMS> b[KC];
#pragma unroll
            for (int t = 0; t < KC; ++t)
                if (t >= ks0) b[t].read(at_r, t, 16 * LC, CA);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < KC; ++t)
                if (t >= ks0) b[t].template add<TERMS>(x, zf[t]);
        }
        if constexpr (LEAN) load_rows(back);
#pragma unroll
        for (int i = 0; i < CT; ++i) {
            de[i] = be * x[i];
            put4<TERMS>(dl + (16 * i + m) * LC + M::place_of(w, g), CA, -in * de[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dv[e] += de[i][e] * to_f32(vv[e][i]);
                db[e] += x[i][e] * ee[e][i];
            }
        }
#pragma unroll
        for (int i = 0; i < CT; ++i) {  // (dY of this lane's own tokens, which it put there)
            const T* mine = yl + (16 * i + m) * LC + M::place_of(w, g);
            const f32x4 x = {to_f32(mine[0]), to_f32(mine[1]), to_f32(mine[2]), to_f32(mine[3])};
            put4<TERMS>(wl + (16 * i + m) * LC + M::place_of(w, g), CA, p.scale * in * x);
        }
        if (c > 0) share_dy();
        const float now = all;
        const float dot = state_dot();
        if constexpr (!LEAN) {
            load_z(back);
            load_values(back, last);
            load_after(back);
        }
        load_gates(back);
        load_dy(c > 1, end == 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float x[CT];
#pragma unroll
            for (int i = 0; i < CT; ++i) x[i] = de[i][e];
            dr.store<CT, T>(yat[e], x);
            if constexpr (TERMS > 1) {
#pragma unroll
                for (int i = 0; i < CT; ++i) x[i] -= (float)(T)x[i];
                lr.store<CT, T>(yat[e], x);
            }
            dv[e] = sum16(dv[e]);
            db[e] = sum16(db[e]);
        }
        if (m == 0) {
            st16(p.dot_v + (at * blocks + cb) * kC + row0, __builtin_bit_cast(uint4, dv));
            st16(p.dot_b + (at * blocks + cb) * kC + row0, __builtin_bit_cast(uint4, db));
        }
        if (lane == 0) p.dot_s[(at * blocks + cb) * kWaves + w] = dot;
        lds_barrier();  // -e^g dE is there, B dU is free
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < CT; ++i) st[t][i] *= now;
#pragma unroll
        for (int k = 0; k < KC; ++k) {
            Operands<T, CT, TERMS> b, y;
            b.read(at_d, k, 16 * LC, CA);
            y.read(at_w, k, 16 * LC, CA);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const Frag kt = columns_of(kl, LS, 16 * (rows.tile0 + t), k, m, g), qt = columns_of(ql, LS, 16 * (rows.tile0 + t), k, m, g);
                b.template add<1>(st[t], &kt);
                y.template add<1>(st[t], &qt);
            }
        }
        lds_barrier();  // K and Q are free
        rows.template share<TERMS>(st, sl, LS, SA);
    }
    // (its addresses computed here, not kept in registers through the chunks)
    int end_lane = threadIdx.x % kWave;
    asm volatile("" : "+v"(end_lane));
    const StateRows<N, CT> ends(w, end_lane);
    if (p.dinit) ends.store(st, p.dinit + (s * p.H + h) * NP + cb * kCols, p.P);
    if (p.init && chunks > 0) {
        ends.load(after, p.init + (s * p.H + h) * NP + cb * kCols, p.P);
        const float dot = state_dot();
        if (end_lane == 0) p.dot_0[((s * p.H + h) * blocks + cb) * kWaves + w] = dot;
    }
}

template <typename T, int N, int CT>
int launch_back(const DeltaParams& p, hipStream_t stream) {
    using M = Mat<T>;
    const int64_t units = p.nseq * p.H * (p.P / p.cols), per = (units + 7) / 8;
    constexpr int LS = N + M::kPad, cols = 16 * CT, states = M::kTerms * cols * LS, rows = 2 * kC * LS;
    constexpr int lds = ((states > rows ? states : rows) + (3 * M::kTerms + 1) * cols * (kC + M::kPad)) * (int)sizeof(T);
    if (hipFuncSetAttribute(reinterpret_cast<const void*>(&delta_back_kernel<T, N, CT>), hipFuncAttributeMaxDynamicSharedMemorySize, lds) != hipSuccess)
        return -1;
    hipLaunchKernelGGL((delta_back_kernel<T, N, CT>), dim3((unsigned)(8 * per)), dim3(kThreads), lds, stream, p, units, per);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

// dq and dk of one chunk and key head, summed over its value heads in registers (no atomics), and their dlog a and dbeta.
// Eight waves.  A wave has 16 rows n of dq^T and dk^T, of all 64 tokens as columns (of fewer where there are fewer
// rows), and of the score tiles those of 16 tokens, either the ones with dY or the ones with dE.  dq and dk are of the inputs' type: in
// bf16 every computed operand (U, dE, the states, the decayed scores) has two terms, 2^-16 of it, which leaves dq and dk their own
// rounding (errors of 1.66e-3; 2.4e-3 with one term of all but U).
//
// 8 x 2048 tokens, 24 heads of 128 by 64, bf16: 309 us, 893 MB read and 227 written (3.6 TB/s): bytes, most of them the fp32 states, e and
// the two-term operands that the passes before made (245 us and 150 MB less to read with one term).  128 registers a lane, for two workgroups a CU, leave
// bf16 no room for loads ahead: the states' rows asked for before the scores, under which they come in fp32 (901 tokens, 6/2 heads of 64 by 32:
// 34.5 us for 37), have 12 registers spilled and take 329 us (64 by 64: 173 us for 165).
template <typename T, int N, int PK>
__global__ void __launch_bounds__(2 * kThreads, sizeof(T) == 2 ? 4 : 2) delta_grad_kernel(DeltaParams p) {
    using M = Mat<T>;
    using Frag = typename M::Frag;
    constexpr int KC = kC / M::kK, KP = PK / M::kK, NTILES = N / 16, CW = NTILES / 2;  // CW: column tiles of a wave (4, 2, 1)
    constexpr int LP = PK + M::kPad, LC = kC + M::kPad, LS = N + M::kPad;
    constexpr int PER = kC * (PK / 4) / (2 * kThreads), FRAGS = kC * N / M::kE / kWave, ROWS = (FRAGS + 7) / 8;
    // dY, dE and U (the latter of TU terms) of a block of value dimensions [token][p], and in the same place the three score matrices
    // [token][contraction] of TU terms; K and Q [token][n].  Keys of 128 leave room for five of six terms beside a second workgroup
    // on the CU: the last one goes in when the first ones have been read
    constexpr int TU = sizeof(T) == 2 ? 2 : 1;
    constexpr bool LATE = TU == 2 && N == 128;
    constexpr int kOperands = (1 + 2 * TU) * kC * LP, kScores = (3 * TU - LATE) * kC * LC;
    __shared__ __attribute__((aligned(16))) T mem[kOperands > kScores ? kOperands : kScores];
    extern __shared__ __attribute__((aligned(16))) char more[];
    __shared__ float ghi[kC], glo[kC];
    T *const yl = mem, *const el = mem + kC * LP, *const ul = mem + (1 + TU) * kC * LP;
    T *const bq = mem, *const bk = mem + TU * kC * LC, *const bqk = mem + 2 * TU * kC * LC;
    T *const kl = reinterpret_cast<T*>(more), *const ql = kl + kC * LS;

    const int64_t slot = blockIdx.x / p.G;
    const int grp = blockIdx.x % p.G, group = p.H / p.G;
    int tid = threadIdx.x, lane = tid % kWave, m = lane % 16, g = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int64_t rows_at = (slot * p.G + grp) * (int64_t)(N * kC);
    uint4 rows[2][ROWS];  // (on their way while the slot's sequence is looked for)
    {
        const Block kb(static_cast<const T*>(p.kr) + rows_at, FRAGS * kWave * 16), qb(static_cast<const T*>(p.qr) + rows_at, FRAGS * kWave * 16);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            rows[0][i] = kb.load16(threadIdx.x * 16, i * 2 * kThreads * 16);
            rows[1][i] = qb.load16(threadIdx.x * 16, i * 2 * kThreads * 16);
        }
    }
    const int64_t s = seq_of_slot(p, slot);
    const Span span = span_of(p, s);
    const int64_t chunk = slot - (span.lo / kC + s);
    if (chunk < 0 || chunk * kC >= span.len) return;
    const int64_t tok0 = span.lo + chunk * kC, HP = (int64_t)p.H * p.P;
    const int have = (int)(span.len - chunk * kC < kC ? span.len - chunk * kC : kC);
    const int w = wave % 4, set = wave / 4;                        // scores: tokens 16 w .., of dY (0) or dE (1)
    const int n0 = 16 * (wave % NTILES), c0 = wave / NTILES * CW;  // products: rows n0 .., column tiles c0 ..
    const int blocks = p.P / p.cols;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int f = wave + i * 8;
        if (FRAGS % 8 != 0 && f >= FRAGS) continue;
        const int at = (16 * (f / (N / M::kK)) + m) * LS + f % (N / M::kK) * M::kK + g * M::kE;
        st16(kl + at, rows[0][i]);
        st16(ql + at, rows[1][i]);
    }
    f32x4 dq[CW], dk[CW];
#pragma unroll
    for (int i = 0; i < CW; ++i) dq[i] = dk[i] = f32x4{};

    // (what follows computes its lane's addresses anew from here: kept through the loops, they would take registers that
    // are not there)
    const auto fresh = [&] {
        asm volatile("" : "+v"(tid));
        lane = tid % kWave;
        m = lane % 16;
        g = lane / 16;
    };
    for (int r = 0; r < group; ++r) {
        const int h = grp * group + r;
        const int64_t at = slot * p.H + h;
        fresh();
        const Block gates(p.gates + at * (kDeltaGates * kC));
        if (tid < kC) {
            ghi[tid] = gates.loadf(tid * 4, kGateHigh * kC * 4);
            glo[tid] = gates.loadf(tid * 4, kGateLow * kC * 4);
        }
        // scores, rows: contraction index j or l; columns: tokens i = 16 w ..  Tiles before w: x_i.u_j, after w: x_l.u_i,
        // tile w: both, the latter in diag; x = dy or de
        f32x4 near[4], diag{};
#pragma unroll
        for (int i = 0; i < 4; ++i) near[i] = f32x4{};
        for (int p0 = 0; p0 < p.P; p0 += PK) {
            fresh();
            uint32_t put[PER], token[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int x = tid + i * 2 * kThreads, t = x / (PK / 4), c = 4 * (x % (PK / 4));
                put[i] = t * LP + c;
                token[i] = (uint32_t)(t * HP + c);
            }
            // everything that the block needs of memory, on its way at once
            const uint32_t bytes = (uint32_t)((have - 1) * HP + PK);
            const int64_t o = tok0 * HP + h * p.P + p0;
            const Block yb(static_cast<const T*>(p.dy) + o, bytes * sizeof(T)), eb(static_cast<const T*>(p.dv) + o, bytes * sizeof(T)), ub(p.wrong + o, bytes * 4);
            typedef typename std::conditional<sizeof(T) == 4, uint4, uint2>::type four;  // four elements
            four x4[1 + TU][PER];
            const Block rb(static_cast<const T*>(TU == 2 ? p.dv_rest : p.dv) + o, bytes * sizeof(T));
            uint4 u4[PER];
            float beta[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if constexpr (sizeof(T) == 4) {
                    x4[0][i] = yb.load16(token[i] * 4, 0);
                    x4[1][i] = eb.load16(token[i] * 4, 0);
                } else {
                    x4[0][i] = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(yb.r, (int)(token[i] * 2), 0, 0));
                    x4[1][i] = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(eb.r, (int)(token[i] * 2), 0, 0));
                    x4[2][i] = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rb.r, (int)(token[i] * 2), 0, 0));
                }
                u4[i] = ub.load16(token[i] * 4, 0);
                beta[i] = gates.loadf(tid / (PK / 4) * 4, (kGateBeta * kC + i * 2 * kThreads / (PK / 4)) * 4);
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                *reinterpret_cast<four*>(yl + put[i]) = x4[0][i];
#pragma unroll
                for (int u = 0; u < TU; ++u) *reinterpret_cast<four*>(el + u * kC * LP + put[i]) = x4[1 + u][i];
                put4<TU>(ul + put[i], kC * LP, beta[i] * as_f32x4(u4[i]));
            }
            const Block sb(p.states + ((slot + s) * p.H + h) * (int64_t)N * p.P + p0);
            const uint32_t sat = (uint32_t)((n0 + m) * p.P + g * M::kE);
            f32x4 x0[KP][M::kE / 4];
            Frag f0[KP][TU], f1[KP][TU];
            const auto load_before = [&] {
#pragma unroll
                for (int k = 0; k < KP; ++k)
#pragma unroll
                    for (int e = 0; e < M::kE / 4; ++e) x0[k][e] = as_f32x4(sb.load16(sat * 4, (k * M::kK + 4 * e) * 4));
            };
            const auto load_after = [&] {
#pragma unroll
                for (int u = 0; u < TU; ++u) {
                    const Block db(static_cast<const T*>(u == 0 ? p.dstates : p.dstates_rest) + at * (int64_t)N * p.P + p0);
#pragma unroll
                    for (int k = 0; k < KP; ++k) f1[k][u] = db.frag<T>(sat * sizeof(T), k * M::kK * sizeof(T));
                }
            };
            if constexpr (TU == 1) {
                load_before();
                load_after();
            }
            __syncthreads();
            // term u of a tile's rows
            const auto row = [&](const T* x, int u, int tile, int k) { return frag(x + u * kC * LP + (16 * tile + m) * LP + k * M::kK + g * M::kE); };
            const auto scores = [&](const T* xl, auto terms) {
                constexpr int TX = decltype(terms)::value;
#pragma unroll
                for (int k = 0; k < KP; ++k) {
                    Frag xi[TX], ui[TU];
#pragma unroll
                    for (int u = 0; u < TX; ++u) xi[u] = row(xl, u, w, k);
#pragma unroll
                    for (int u = 0; u < TU; ++u) ui[u] = row(ul, u, w, k);
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        // (the tile's own rows: U's where they come before, dY's or dE's where after)
                        const bool up = t <= w;
                        const T* own = up ? ul : xl;
                        const Frag x = row(own, 0, t, k);
                        if constexpr (TU == 2) {
                            const Frag rest = row(up || TX == 2 ? own + kC * LP : own, 0, t, k);
                            near[t] = M::mma(rest, up ? xi[0] : ui[TX == 2 ? 0 : 1], near[t]);
                            if constexpr (TX == 2) near[t] = M::mma(x, up ? xi[1] : ui[1], near[t]);
                        }
                        near[t] = M::mma(x, up ? xi[0] : ui[0], near[t]);
                        if (TU == 2 || t % 2 == 1) __builtin_amdgcn_sched_barrier(0);
                    }
#pragma unroll
                    for (int v = TX - 1; v >= 0; --v)
#pragma unroll
                        for (int u = TU - 1; u >= 0; --u)
                            if (u + v < TU) diag = M::mma(xi[v], ui[u], diag);
                    __builtin_amdgcn_sched_barrier(0);  // (here and below: the operands of one step at a time, in 128 registers)
                }
            };
            if constexpr (TU == 1) scores(set == 0 ? yl : el, std::integral_constant<int, 1>{});
            else if (set == 0) scores(yl, std::integral_constant<int, 1>{});
            else scores(el, std::integral_constant<int, TU>{});
            // products with the states before and after the chunk
            if constexpr (TU > 1) load_before();
#pragma unroll
            for (int k = 0; k < KP; ++k)
#pragma unroll
                for (int e = 0; e < M::kE; ++e) {
                    float rest = x0[k][e / 4][e % 4];
#pragma unroll
                    for (int u = 0; u < TU; ++u) {
                        f0[k][u][e] = (T)rest;
                        rest -= (float)f0[k][u][e];
                    }
                }
#pragma unroll
            for (int i = 0; i < CW; ++i) {
                f32x4 a{}, b{};
#pragma unroll
                for (int k = 0; k < KP; ++k) {
                    const Frag y = row(yl, 0, c0 + i, k);
#pragma unroll
                    for (int u = TU - 1; u >= 0; --u) a = M::mma(f0[k][u], y, a);
#pragma unroll
                    for (int v = TU - 1; v >= 0; --v) {
                        const Frag x = row(el, v, c0 + i, k);
#pragma unroll
                        for (int u = TU - 1; u >= 0; --u)
                            if (u + v < TU) b = M::mma(f0[k][u], x, b);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                const float in = gates.loadf((16 * c0 + m) * 4, (kGateIn * kC + 16 * i) * 4);
                dq[i] += (p.scale * in) * a;
                dk[i] -= in * b;
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (TU > 1) load_after();
#pragma unroll
            for (int i = 0; i < CW; ++i) {
                f32x4 c{};
#pragma unroll
                for (int k = 0; k < KP; ++k) {
#pragma unroll
                    for (int v = TU - 1; v >= 0; --v) {
                        const Frag x = row(ul, v, c0 + i, k);
#pragma unroll
                        for (int u = TU - 1; u >= 0; --u)
                            if (u + v < TU) c = M::mma(f1[k][u], x, c);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                dk[i] += gates.loadf((16 * c0 + m) * 4, (kGateOut * kC + 16 * i) * 4) * c;
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        __syncthreads();
        fresh();
        uint2 late[LATE ? 4 : 1];  // the second terms of bqk
        {
            const int i = 16 * w + m;
            const float hi = ghi[i], li = glo[i], by = set == 0 ? p.scale : -1.f;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                f32x4 before{}, after{};  // of contraction indices up to i, and from i on
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = 16 * t + 4 * g + e;
                    const float apart = (hi - ghi[j]) + (li - glo[j]);  // of i > j; for j > i the decay is of its opposite
                    const float far = j <= i ? apart : -apart, d = by * (sizeof(T) == 4 ? expf(far) : __expf(far));
                    if (j < i || (set == 0 && j == i)) before[e] = d * near[t][e];
                    if (j > i || (set == 0 && j == i)) after[e] = d * (t == w ? diag[e] : near[t][e]);
                }
                const int o = i * LC + M::place_of(t, g);
                if (set == 0) {
                    put4<TU>(bq + o, kC * LC, before);
                    put4<LATE ? 1 : TU>(bqk + o, kC * LC, after);
                    if constexpr (LATE) {
                        float x[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[e] = after[e] - (float)(T)after[e];
                        late[t].x = take2(x[0], x[1]);
                        late[t].y = take2(x[2], x[3]);
                    }
                } else {
                    put4<TU>(bk + o, kC * LC, before + after);
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < KC; ++k) {
            const Frag kf = columns_of(kl, LS, n0, k, m, g), qf = columns_of(ql, LS, n0, k, m, g);
#pragma unroll
            for (int i = 0; i < CW; ++i) {
                const int o = (16 * (c0 + i) + m) * LC + k * M::kK + g * M::kE;
#pragma unroll
                for (int u = TU - 1; u >= 0; --u) {
                    dq[i] = M::mma(kf, frag(bq + u * kC * LC + o), dq[i]);
                    dk[i] = M::mma(kf, frag(bk + u * kC * LC + o), dk[i]);
                    if (u == 0 || !LATE) dk[i] = M::mma(qf, frag(bqk + u * kC * LC + o), dk[i]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if constexpr (LATE) {
            __syncthreads();
            if (set == 0) {
#pragma unroll
                for (int t = 0; t < 4; ++t) st8(mem + (16 * w + m) * LC + M::place_of(t, g), late[t]);
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < KC; ++k) {
                const Frag qf = columns_of(ql, LS, n0, k, m, g);
#pragma unroll
                for (int i = 0; i < CW; ++i) {
                    dk[i] = M::mma(qf, frag(mem + (16 * (c0 + i) + m) * LC + k * M::kK + g * M::kE), dk[i]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        if (wave == r % 8) {
            // the sums, token by token; of the decays from a token to the chunk's end
            double db = 0.0, dg = 0.0;
            for (int b = 0; b < blocks; ++b) {
                const int64_t o = (at * blocks + b) * kC + lane;
                db += p.dot_b[o];
                dg += (double)p.dot_y[o] - p.dot_v[o];
            }
            const int parts = blocks * kWaves;
            double all = lane < parts ? p.dot_s[at * parts + lane] : 0.0, before = 0.0;
            if (lane < parts && chunk > 0) before = p.dot_s[(at - p.H) * parts + lane];
            if (lane < parts && chunk == 0 && p.init) before = p.dot_0[(s * p.H + h) * parts + lane];
#pragma unroll
            for (int off = 1; off < kWave; off <<= 1) {
                const double o = __shfl_down(dg, off, kWave);
                if (lane + off < kWave) dg += o;
                all += __shfl_xor(all, off, kWave);
                before += __shfl_xor(before, off, kWave);
            }
            const double missing = before - all - __shfl(dg, 0, kWave);
            int rows = have;
            asm volatile("" : "+v"(rows));  // (widened here, not kept in registers through the heads)
            if (lane < have) {
                const int64_t o = (tok0 + lane) * p.H + h;
                p.dbeta[o] = (float)db;
                // (a decay of zero passes nothing on; the sums would leave their rounding)
                p.dlog_a[o] = expf(p.log_a[o]) == 0.f ? 0.f : (float)(dg + all + missing * (1.0 - (double)lane / rows));
            }
        }
    }
    // by way of LDS, in the place of K and Q: rows of N elements leave whole
    fresh();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < CW; ++i) {
        const int at = (16 * (c0 + i) + m) * LS + n0 + 4 * g;
        store4(ql + at, dq[i][0], dq[i][1], dq[i][2], dq[i][3]);
        store4(kl + at, dk[i][0], dk[i][1], dk[i][2], dk[i][3]);
    }
    __syncthreads();
    for (int f = tid; f < have * (N / M::kE); f += 2 * kThreads) {
        const int t = f / (N / M::kE), c = f % (N / M::kE) * M::kE;
        const int64_t o = ((tok0 + t) * p.G + grp) * N + c;
        st16(static_cast<T*>(p.dq) + o, ld16(ql + t * LS + c));
        st16(static_cast<T*>(p.dk) + o, ld16(kl + t * LS + c));
    }
}

template <typename T, int N, int PK>
int launch_grad(const DeltaParams& p, hipStream_t stream) {
    constexpr int lds = 2 * kC * (N + Mat<T>::kPad) * (int)sizeof(T);
    const auto kernel = &delta_grad_kernel<T, N, PK>;
    if (hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, lds) != hipSuccess) return -1;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(p.slots * p.G)), dim3(2 * kThreads), lds, stream, p);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

template <typename T, int N>
int launch_backward(const DeltaParams& p, hipStream_t stream) {
    int rc = 0;
    if (p.total > 0) {
        rc = launch_prep<T, N, true>(p, stream);
        if (rc == 0) rc = launch_walk<T, N, true>(p, stream);
    }
    if (rc == 0) rc = p.cols == 16 ? launch_back<T, N, 1>(p, stream) : launch_back<T, N, 2>(p, stream);
    if (rc != 0 || p.total == 0) return rc;
    return p.P % 64 == 0 ? launch_grad<T, N, 64>(p, stream) : launch_grad<T, N, 32>(p, stream);
}

}  // namespace
}  // namespace delta

int launch_delta_backward(const DeltaParams& p, int dtype, hipStream_t stream) {
    switch (p.N) {
        case 32: return dtype == 1 ? delta::launch_backward<__bf16, 32>(p, stream) : delta::launch_backward<float, 32>(p, stream);
        case 64: return dtype == 1 ? delta::launch_backward<__bf16, 64>(p, stream) : delta::launch_backward<float, 64>(p, stream);
        case 128: return dtype == 1 ? delta::launch_backward<__bf16, 128>(p, stream) : delta::launch_backward<float, 128>(p, stream);
        default: return -2;
    }
}

}  // namespace ssd
