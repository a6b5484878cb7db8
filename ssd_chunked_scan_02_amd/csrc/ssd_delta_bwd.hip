// The backward pass of the gated delta rule, gfx950.  With the notation of ssd_delta_walk.h, x the gradient that reaches
// U = B E, and dS' the gradient of the state after a chunk:
//     dU = scale P^T dY + e^(gC - g) (K dS'),  x = dU + Z^T B dU,  dE = B x = dV,
//     dS = e^gC dS' + scale Q^T (e^g dY) - K^T (e^g dE),
//     dbeta_i = x_i . e_i,
//     dlog a_t = sum over i >= t of (dy_i . y_i - dv_i . v_i), plus <dS', S'>
// (the sums of what each token's decay multiplies, row by row and column by column, telescoped), and
//     dq_i = scale (e^g_i S dy_i + sum_{j<=i} D_ij (dy_i.u_j) k_j)
//     dk_i = scale sum_{l>=i} D_li (dy_l.u_i) q_l - sum_{l>i} D_li (de_l.u_i) k_l - sum_{j<i} D_ij (de_i.u_j) k_j
//            + e^(gC - g_i) dS' u_i - e^g_i S de_i.
// Four launches: delta_prep_kernel and delta_walk_kernel again (which keep the states before the chunks, e and dy . y),
// delta_back_kernel down the chunks from the last one, delta_grad_kernel for dq, dk and the sums, all chunks at once.
#include "ssd_delta_prep.h"
#include "ssd_delta_walk.h"

namespace ssd {
namespace delta {
namespace {

// The gradient of the state, from chunk to chunk towards the first: as delta_walk_kernel, 32 columns a workgroup, the
// rows split over its waves, every product of fp32 values on operands of all terms.
template <typename T, int N>
__global__ void __launch_bounds__(kThreads, N * sizeof(T) >= 256 ? 1 : 2) delta_back_kernel(DeltaParams p, int64_t units, int64_t per_xcd) {
    using M = Mat<T>;
    using Frag = typename M::Frag;
    constexpr int KN = N / M::kK, KC = kC / M::kK, TERMS = M::kTerms, NT = StateRows<N>::NT;
    constexpr int LS = N + M::kPad, LC = kC + M::kPad, SA = kCols * LS, CA = kCols * LC;
    // dS' [column][n]; dY [column][token]; of all terms: scale e^g dY, for this chunk and the next, B dU, -e^g dE
    __shared__ __attribute__((aligned(16))) T sl[TERMS * SA];
    __shared__ __attribute__((aligned(16))) T yl[CA];
    extern __shared__ __attribute__((aligned(16))) char more[];
    T* const wl = reinterpret_cast<T*>(more);
    T* const rl = wl + 2 * TERMS * CA;
    T* const dl = rl + TERMS * CA;

    const int64_t unit = xcd_work_index(blockIdx.x, per_xcd, units);
    if (unit < 0) return;
    const int blocks = p.P / kCols, cb = (int)(unit % blocks), h = (int)(unit / blocks % p.H), grp = h / (p.H / p.G);
    const int64_t s = unit / blocks / p.H;
    const Span span = span_of(p, s);
    const int64_t slot0 = span.lo / kC + s, chunks = (span.len + kC - 1) / kC;
    const int lane = threadIdx.x % kWave, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), m = lane % 16, g = lane / 16;
    const int row0 = 16 * w + 4 * g, ks0 = 16 * w / M::kK;  // (steps before ks0 are left of the diagonal: zero)
    const StateRows<N> rows(w, lane);
    const int64_t NP = (int64_t)N * p.P, HP = (int64_t)p.H * p.P, vcol = (int64_t)h * p.P + cb * kCols;

    f32x4 st[NT][CT];
    rows.load(st, p.dfinal ? p.dfinal + (s * p.H + h) * NP + cb * kCols : nullptr, p.P);
    rows.template share<TERMS>(st, sl, LS, SA);

    Frag kf[KN], zf[KC][TERMS], pf[KC][TERMS], tf[NT][KC], uf[NT][KC];
    f32x4 in, out, be, ahead, after[NT][CT];  // ahead: e^g of the chunk whose dY is loaded
    float all;
    T vv[4][CT], yv[4][CT];
    float ee[4][CT];
    const auto have_of = [&](int64_t c) { return span.len - c * kC < kC ? span.len - c * kC : (int64_t)kC; };
    const auto load_rows = [&](int64_t c) {
        const Rows<T> kr(static_cast<const T*>(p.k) + (span.lo + c * kC) * p.k_stride + grp * N, have_of(c), p.k_stride, N);
#pragma unroll
        for (int i = 0; i < KN; ++i) kf[i] = kr.frag(16 * w + m, i * M::kK + g * M::kE);
        const T* sc = static_cast<const T*>(p.scores_t) + ((slot0 + c) * p.H + h) * (int64_t)(TERMS * kC * kC) + (w * KC * kWave + lane) * M::kE;
#pragma unroll
        for (int i = 0; i < KC; ++i)
#pragma unroll
            for (int u = 0; u < TERMS; ++u) pf[i][u] = frag(sc + u * (kC * kC) + max(i, ks0) * (kWave * M::kE));
    };
    const auto load_z = [&](int64_t c) {
        const T* z = static_cast<const T*>(p.zt) + ((slot0 + c) * p.H + h) * (int64_t)(TERMS * kC * kC) + (w * KC * kWave + lane) * M::kE;
#pragma unroll
        for (int i = 0; i < KC; ++i)
#pragma unroll
            for (int u = 0; u < TERMS; ++u) zf[i][u] = frag(z + u * (kC * kC) + max(i, ks0) * (kWave * M::kE));
    };
    const auto load_values = [&](int64_t c) {
        const float* gates = p.gates + ((slot0 + c) * p.H + h) * (kDeltaGates * kC);
        in = as_f32x4(ld16(gates + kGateIn * kC + row0));
        out = as_f32x4(ld16(gates + kGateOut * kC + row0));
        be = as_f32x4(ld16(gates + kGateBeta * kC + row0));
        all = gates[kGateIn * kC + kC - 1];
        const int64_t t0 = span.lo + c * kC;
        const Rows<T> vr(static_cast<const T*>(p.v) + t0 * p.v_stride + vcol, have_of(c), p.v_stride, kCols);
        const Rows<float> er(p.wrong + t0 * HP + vcol, have_of(c), HP, kCols);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            vr.load2(row0 + e, 2 * m, vv[e]);
            er.load2(row0 + e, 2 * m, ee[e]);
        }
    };
    const auto load_rest = [&](int64_t c) {
        const int64_t o = ((slot0 + c) * p.G + grp) * (int64_t)(N * kC) + (rows.tile0 * KC * kWave + lane) * M::kE;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < KC; ++i) {
                tf[t][i] = frag(static_cast<const T*>(p.kt) + o + (t * KC + i) * (kWave * M::kE));
                uf[t][i] = frag(static_cast<const T*>(p.qt) + o + (t * KC + i) * (kWave * M::kE));
            }
    };
    const auto load_after = [&](int64_t c) { rows.load(after, p.states + ((slot0 + c + 1 + s) * p.H + h) * NP + cb * kCols, p.P); };
    const auto load_dy = [&](int64_t c) {
        const Rows<T> yr(static_cast<const T*>(p.dy) + (span.lo + c * kC) * HP + vcol, have_of(c), HP, kCols);
#pragma unroll
        for (int e = 0; e < 4; ++e) yr.load2(row0 + e, 2 * m, yv[e]);
        ahead = as_f32x4(ld16(p.gates + ((slot0 + c) * p.H + h) * (kDeltaGates * kC) + kGateIn * kC + row0));
    };
    const auto share_dy = [&](T* to) {
#pragma unroll
        for (int i = 0; i < CT; ++i) {
            const f32x4 x = {to_f32(yv[0][i]), to_f32(yv[1][i]), to_f32(yv[2][i]), to_f32(yv[3][i])};
            put4<1>(yl + (16 * i + m) * LC + M::place_of(w, g), 0, x);
            put4<TERMS>(to + (16 * i + m) * LC + M::place_of(w, g), CA, p.scale * ahead * x);
        }
    };
    if (chunks > 0) {
        const int64_t c = chunks - 1;
        load_dy(c);
        load_rows(c);
        load_z(c);
        load_values(c);
        load_rest(c);
        load_after(c);
        share_dy(wl + (c & 1) * (TERMS * CA));
        load_dy(c > 0 ? c - 1 : 0);
    }
    for (int64_t c = chunks - 1; c >= 0; --c) {
        const int64_t next = c > 0 ? c - 1 : 0, at = (slot0 + c) * p.H + h;
        float dot = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < CT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) dot += st[t][i][e] * after[t][i][e];
        if (StateRows<N>::kAll || rows.own) {
            const Rows<T> sr(static_cast<T*>(p.dstates) + at * NP + cb * kCols, N, p.P, kCols);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) sr.store2(16 * (rows.tile0 + t) + 4 * g + e, 2 * m, st[t][0][e], st[t][1][e]);
        } else {
            dot = 0.f;
        }
        lds_barrier();  // dS' and dY are there
        f32x4 x[CT];
#pragma unroll
        for (int i = 0; i < CT; ++i) {
            f32x4 a{}, b{};
#pragma unroll
            for (int t = 0; t < KN; ++t) a = mma_terms<T, 1, TERMS>(&kf[t], sl + (16 * i + m) * LS + t * M::kK + g * M::kE, SA, a);
#pragma unroll
            for (int t = 0; t < KC; ++t)
                if (t >= ks0) b = mma_terms<T, TERMS, 1>(pf[t], yl + (16 * i + m) * LC + t * M::kK + g * M::kE, 0, b);
            x[i] = p.scale * b + out * a;
            put4<TERMS>(rl + (16 * i + m) * LC + M::place_of(w, g), CA, be * x[i]);
        }
        load_rows(next);
        lds_barrier();  // B dU is there, dS' and dY are free
        f32x4 dv{}, db{};
        const Rows<T> dr(static_cast<T*>(p.dv) + (span.lo + c * kC) * HP + vcol, have_of(c), HP, kCols);
        f32x4 de[CT];
#pragma unroll
        for (int i = 0; i < CT; ++i) {
#pragma unroll
            for (int t = 0; t < KC; ++t)
                if (t >= ks0) x[i] = mma_terms<T, TERMS, TERMS>(zf[t], rl + (16 * i + m) * LC + t * M::kK + g * M::kE, CA, x[i]);
            de[i] = be * x[i];
            put4<TERMS>(dl + (16 * i + m) * LC + M::place_of(w, g), CA, -in * de[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dv[e] += de[i][e] * to_f32(vv[e][i]);
                db[e] += x[i][e] * ee[e][i];
            }
        }
        if (c > 0) share_dy(wl + (next & 1) * (TERMS * CA));
        const float now = all;
        load_z(next);
        load_values(next);
        load_after(next);
        load_dy(next > 0 ? next - 1 : 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            dr.store2(row0 + e, 2 * m, de[0][e], de[1][e]);
            dv[e] = sum16(dv[e]);
            db[e] = sum16(db[e]);
        }
        if (m == 0) {
            st16(p.dot_v + (at * blocks + cb) * kC + row0, __builtin_bit_cast(uint4, dv));
            st16(p.dot_b + (at * blocks + cb) * kC + row0, __builtin_bit_cast(uint4, db));
        }
        dot = sum16(dot);
        dot += __shfl_xor(dot, 16, kWave);
        dot += __shfl_xor(dot, 32, kWave);
        if (lane == 0) p.dot_s[(at * blocks + cb) * kWaves + w] = dot;
        lds_barrier();  // -e^g dE is there, B dU is free
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < CT; ++i) {
                st[t][i] *= now;
#pragma unroll
                for (int k = 0; k < KC; ++k) {
                    const int o = (16 * i + m) * LC + k * M::kK + g * M::kE;
                    st[t][i] = mma_terms<T, 1, TERMS>(&tf[t][k], dl + o, CA, st[t][i]);
                    st[t][i] = mma_terms<T, 1, TERMS>(&uf[t][k], wl + (c & 1) * (TERMS * CA) + o, CA, st[t][i]);
                }
            }
        rows.template share<TERMS>(st, sl, LS, SA);
        load_rest(next);
    }
    if (p.dinit) rows.store(st, p.dinit + (s * p.H + h) * NP + cb * kCols, p.P);
}

template <typename T, int N>
int launch_back(const DeltaParams& p, hipStream_t stream) {
    using M = Mat<T>;
    const int64_t units = p.nseq * p.H * (p.P / kCols), per = (units + 7) / 8;
    constexpr int lds = 4 * M::kTerms * kCols * (kC + M::kPad) * (int)sizeof(T);
    if (hipFuncSetAttribute(reinterpret_cast<const void*>(&delta_back_kernel<T, N>), hipFuncAttributeMaxDynamicSharedMemorySize, lds) != hipSuccess)
        return -1;
    hipLaunchKernelGGL((delta_back_kernel<T, N>), dim3((unsigned)(8 * per)), dim3(kThreads), lds, stream, p, units, per);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

// dq and dk of one chunk and key head, summed over its value heads in registers (no atomics), and their dlog a and dbeta.
// A wave has a quarter of the rows n of dq^T and dk^T, for all 64 tokens as columns; the score tiles it computes
// are those of its own 16 tokens.  One bf16 term each: the outputs are of the inputs' type.
template <typename T, int N, int PK>
__global__ void __launch_bounds__(kThreads, 2) delta_grad_kernel(DeltaParams p) {
    using M = Mat<T>;
    using Frag = typename M::Frag;
    constexpr int KC = kC / M::kK, KP = PK / M::kK, NT = (N / 16 + 3) / 4;
    constexpr int LP = PK + M::kPad, LC = kC + M::kPad;
    // dY, dE and U of a block of value dimensions [token][p]; then the three score matrices [token][contraction]
    __shared__ __attribute__((aligned(16))) T mem[3 * kC * (LP > LC ? LP : LC)];
    __shared__ float ghi[kC], glo[kC];
    T *const yl = mem, *const el = mem + kC * LP, *const ul = mem + 2 * kC * LP;
    T *const bq = mem, *const bk = mem + kC * LC, *const bqk = mem + 2 * kC * LC;

    const int64_t slot = blockIdx.x / p.G;
    const int grp = blockIdx.x % p.G, group = p.H / p.G;
    const int64_t s = seq_of_slot(p, slot);
    const Span span = span_of(p, s);
    const int64_t chunk = slot - (span.lo / kC + s);
    if (chunk < 0 || chunk * kC >= span.len) return;
    const int64_t tok0 = span.lo + chunk * kC;
    const int have = (int)(span.len - chunk * kC < kC ? span.len - chunk * kC : kC);
    const int lane = threadIdx.x % kWave, w = threadIdx.x / kWave, m = lane % 16, g = lane / 16;
    const int tile0 = w * NT, blocks = p.P / kCols;

    f32x4 dq[NT][4], dk[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) dq[t][i] = dk[t][i] = f32x4{};

    for (int r = 0; r < group; ++r) {
        const int h = grp * group + r;
        const int64_t at = slot * p.H + h;
        const float* gates = p.gates + at * (kDeltaGates * kC);
        __syncthreads();
        if (w == 0) {
            ghi[lane] = gates[kGateHigh * kC + lane];
            glo[lane] = gates[kGateLow * kC + lane];
            // the sums, token by token; of the decays from a token to the chunk's end
            double db = 0.0, dg = 0.0;
            for (int b = 0; b < blocks; ++b) {
                const int64_t o = (at * blocks + b) * kC + lane;
                db += p.dot_b[o];
                dg += (double)p.dot_y[o] - p.dot_v[o];
            }
#pragma unroll
            for (int off = 1; off < kWave; off <<= 1) {
                const double o = __shfl_down(dg, off, kWave);
                if (lane + off < kWave) dg += o;
            }
            for (int b = 0; b < blocks * kWaves; ++b) dg += p.dot_s[at * blocks * kWaves + b];
            if (lane < have) {
                const int64_t o = (tok0 + lane) * p.H + h;
                p.dbeta[o] = (float)db;
                // (a decay of zero passes nothing on; the sums would leave their rounding)
                p.dlog_a[o] = expf(p.log_a[o]) == 0.f ? 0.f : (float)dg;
            }
        }
        float in[4], out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            in[i] = gates[kGateIn * kC + 16 * i + m];
            out[i] = gates[kGateOut * kC + 16 * i + m];
        }
        // rows: contraction index j or l; columns: the wave's own tokens i
        f32x4 near1[4], near2[4], own1{}, own2{};  // tiles before w: dy_i.u_j, de_i.u_j; after w: dy_l.u_i, de_l.u_i
        f32x4 diag1{}, diag2{};                    // tile w: own for j, diag for l
#pragma unroll
        for (int i = 0; i < 4; ++i) near1[i] = near2[i] = f32x4{};
        for (int p0 = 0; p0 < p.P; p0 += PK) {
            __syncthreads();
            for (int i = threadIdx.x; i < kC * (PK / 4); i += kThreads) {
                const int t = i / (PK / 4), c = 4 * (i % (PK / 4));
                f32x4 y{}, e{}, u{};
                if (t < have) {
                    const int64_t o = ((tok0 + t) * p.H + h) * p.P + p0 + c;
                    u = gates[kGateBeta * kC + t] * as_f32x4(ld16(p.wrong + o));
                    if constexpr (sizeof(T) == 4) {
                        y = as_f32x4(ld16(static_cast<const float*>(p.dy) + o));
                        e = as_f32x4(ld16(static_cast<const float*>(p.dv) + o));
                    } else {
                        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
                        const bf16x4 a = *reinterpret_cast<const bf16x4*>(static_cast<const T*>(p.dy) + o);
                        const bf16x4 b = *reinterpret_cast<const bf16x4*>(static_cast<const T*>(p.dv) + o);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            y[k] = (float)a[k];
                            e[k] = (float)b[k];
                        }
                    }
                }
                put4<1>(yl + t * LP + c, 0, y);
                put4<1>(el + t * LP + c, 0, e);
                put4<1>(ul + t * LP + c, 0, u);
            }
            __syncthreads();
            const auto row = [&](const T* x, int tile, int k) { return frag(x + (16 * tile + m) * LP + k * M::kK + g * M::kE); };
#pragma unroll
            for (int k = 0; k < KP; ++k) {
                const Frag yi = row(yl, w, k), ei = row(el, w, k), ui = row(ul, w, k);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if (t < w) {
                        const Frag uj = row(ul, t, k);
                        near1[t] = M::mma(uj, yi, near1[t]);
                        near2[t] = M::mma(uj, ei, near2[t]);
                    } else if (t > w) {
                        near1[t] = M::mma(row(yl, t, k), ui, near1[t]);
                        near2[t] = M::mma(row(el, t, k), ui, near2[t]);
                    }
                }
                own1 = M::mma(ui, yi, own1);
                own2 = M::mma(ui, ei, own2);
                diag1 = M::mma(yi, ui, diag1);
                diag2 = M::mma(ei, ui, diag2);
            }
            // products with the states before and after the chunk
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (tile0 + t >= N / 16) continue;
                const int64_t n = 16 * (tile0 + t) + m;
                const float* s0 = p.states + (((slot + s) * p.H + h) * N + n) * p.P + p0 + g * M::kE;
                const T* s1 = static_cast<const T*>(p.dstates) + (at * N + n) * p.P + p0 + g * M::kE;
                Frag f0[KP], f1[KP];
#pragma unroll
                for (int k = 0; k < KP; ++k) {
                    f1[k] = frag(s1 + k * M::kK);
#pragma unroll
                    for (int e = 0; e < M::kE; e += 4) {
                        const f32x4 x = as_f32x4(ld16(s0 + k * M::kK + e));
#pragma unroll
                        for (int j = 0; j < 4; ++j) f0[k][e + j] = (T)x[j];
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f32x4 a{}, b{}, c{};
#pragma unroll
                    for (int k = 0; k < KP; ++k) {
                        a = M::mma(f0[k], row(yl, i, k), a);
                        b = M::mma(f0[k], row(el, i, k), b);
                        c = M::mma(f1[k], row(ul, i, k), c);
                    }
                    dq[t][i] += (p.scale * in[i]) * a;
                    dk[t][i] += out[i] * c - in[i] * b;
                }
            }
        }
        __syncthreads();
        {
            const int i = 16 * w + m;
            const float hi = ghi[i], li = glo[i];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                f32x4 a{}, b{}, c{};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = 16 * t + 4 * g + e;
                    const float apart = (hi - ghi[j]) + (li - glo[j]);  // of i > j; for j > i the decay is of its opposite
                    const float d = expf(j <= i ? apart : -apart);
                    if (t < w) {
                        a[e] = p.scale * d * near1[t][e];
                        b[e] = -d * near2[t][e];
                    } else if (t > w) {
                        c[e] = p.scale * d * near1[t][e];
                        b[e] = -d * near2[t][e];
                    } else {
                        a[e] = j <= i ? p.scale * d * own1[e] : 0.f;
                        c[e] = j >= i ? p.scale * d * diag1[e] : 0.f;
                        b[e] = j < i ? -d * own2[e] : j > i ? -d * diag2[e] : 0.f;
                    }
                }
                const int o = i * LC + M::place_of(t, g);
                put4<1>(bq + o, 0, a);
                put4<1>(bk + o, 0, b);
                put4<1>(bqk + o, 0, c);
            }
        }
        __syncthreads();
        const T* kt = static_cast<const T*>(p.kt) + (slot * p.G + grp) * (int64_t)(N * kC) + lane * M::kE;
        const T* qt = static_cast<const T*>(p.qt) + (slot * p.G + grp) * (int64_t)(N * kC) + lane * M::kE;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (tile0 + t >= N / 16) continue;
#pragma unroll
            for (int k = 0; k < KC; ++k) {
                const Frag kf = frag(kt + ((tile0 + t) * KC + k) * (kWave * M::kE)), qf = frag(qt + ((tile0 + t) * KC + k) * (kWave * M::kE));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int o = (16 * i + m) * LC + k * M::kK + g * M::kE;
                    dq[t][i] = M::mma(kf, frag(bq + o), dq[t][i]);
                    dk[t][i] = M::mma(kf, frag(bk + o), dk[t][i]);
                    dk[t][i] = M::mma(qf, frag(bqk + o), dk[t][i]);
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if (tile0 + t >= N / 16) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (16 * i + m >= have) continue;
            const int64_t o = ((tok0 + 16 * i + m) * p.G + grp) * N + 16 * (tile0 + t) + 4 * g;
            store4(static_cast<T*>(p.dq) + o, dq[t][i][0], dq[t][i][1], dq[t][i][2], dq[t][i][3]);
            store4(static_cast<T*>(p.dk) + o, dk[t][i][0], dk[t][i][1], dk[t][i][2], dk[t][i][3]);
        }
    }
}

template <typename T, int N>
int launch_backward(const DeltaParams& p, hipStream_t stream) {
    int rc = 0;
    if (p.total > 0) {
        rc = launch_prep<T, N, true>(p, stream);
        if (rc == 0) rc = launch_walk<T, N, true>(p, stream);
    }
    if (rc == 0) rc = launch_back<T, N>(p, stream);
    if (rc != 0 || p.total == 0) return rc;
    if (p.P % 64 == 0) hipLaunchKernelGGL((delta_grad_kernel<T, N, 64>), dim3((unsigned)(p.slots * p.G)), dim3(kThreads), 0, stream, p);
    else hipLaunchKernelGGL((delta_grad_kernel<T, N, 32>), dim3((unsigned)(p.slots * p.G)), dim3(kThreads), 0, stream, p);
    return hipGetLastError() == hipSuccess ? 0 : -1;
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
