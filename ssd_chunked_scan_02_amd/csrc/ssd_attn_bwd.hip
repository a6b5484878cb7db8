// Attention over a packed batch of documents, backward, gfx950.  With p from the forward pass's lse and
// D_i = sum_j p_ij (dy_i . v_j):
//     dS_ij = p_ij (dy_i . v_j - D_i),  dz_ij = dS_ij (1 - tanh^2),
//     dq_i = scale sum_j dz_ij k_j,  dk_j = scale sum_i dz_ij q_i,  dv_j = sum_i p_ij dy_i,
//     dtable[b] = sum of dS over the cells of bucket b.
//
// Two kernels, each owning what it sums, so that nothing is added by atomics and every run gives the
// same bits: attn_dq_kernel owns 128 queries of a head and streams keys (S^T, dP^T, dq^T), and leaves D for
// attn_dkv_kernel, which owns 128 keys of a key head and streams the queries of every head of its group
// (S, dP, dv^T, dk^T).  That is 7 products where sharing S and dP would need 5, and no partial
// gradients through memory.  Both keep their rows' operands and gradients in registers; the tile layout
// and operand order are the forward kernel's (ssd_attn_common.h).
//
// D is sum_d dy_id y_id, which is as exact as the given y.  The gradient of the table sums dS over whole
// diagonals, where the error of a bf16 y would be most of the result's, so with a table gradient the
// query kernel takes D from its definition in a first pass over the keys.
#include "ssd_attn_common.h"

namespace ssd {
namespace attn {
namespace {

constexpr int kDiagRows = 16;                   // keys of a staged block of dS
constexpr int kDiagStride = 33;                 // its row stride: 32 queries, and 1 against bank conflicts
constexpr int kDiagBlock = kDiagRows * kDiagStride;

// LDS of the bias, after the tiles: the head's bias by relative position, and with a table gradient a
// block of dS and sums by relative position for each wave.
__host__ __device__ inline int bias_floats(int bias, int md, bool grad) {
    if (bias != kBiasBuckets) return 0;
    const int reach = 2 * md + 1;
    return reach + (grad ? kWaves * (reach + kDiagBlock) + 2 * kWaves : 0);
}

// Sum of a bucket's cells over the sums by relative position (a wave's array, interior only: distances of
// max_distance and more are summed apart).
__device__ __forceinline__ float fold_bucket(const AttnBuckets& b, const float* sums, int bucket) {
    const int n = b.nborders + 1, in = bucket % n;
    const bool behind = b.both && bucket >= n;
    const int lo = in == 0 ? 0 : b.borders[in - 1], hi = in == n - 1 ? b.max_distance : b.borders[in];
    float v = 0.f;
    for (int d = behind && lo == 0 ? 1 : lo; d < hi; ++d) v += sums[b.max_distance + (behind ? d : -d)];
    if (!b.both && in == 0)
        for (int d = 1; d < b.max_distance; ++d) v += sums[b.max_distance + d];
    return v;
}

template <typename T, int D, bool CAP, int BIAS>
__global__ void __launch_bounds__(kThreads, 2) attn_dq_kernel(AttnParams p) {
    using O = Op<T>;
    using L = Tile<T, D>;
    using Frag = typename O::Frag;
    constexpr int KT = O::kKT, NS = KT / 32, NT = D / O::kK, DT = D / 32, PK = 32 / O::kK;
    __shared__ __attribute__((aligned(16))) T ks[2][L::kElems];
    __shared__ __attribute__((aligned(16))) T vs[2][L::kElems];
    extern __shared__ float extra[];

    int slot, head;
    work_item(blockIdx.x, p.q_slots, p.H, slot, head);
    const Span sp = find_span(p, slot, false);
    const bool grad = BIAS == kBiasBuckets && p.dtable != nullptr;
    float* part = grad ? p.table_part + ((int64_t)slot * p.H + head) * p.bk.total : nullptr;
    if (sp.tile < 0) {
        if (grad)
            for (int i = threadIdx.x; i < p.bk.total; i += kThreads) part[i] = 0.f;
        return;
    }
    const int kvh = head / (p.H / p.Hk);
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, half = lane / 32;
    const int shift = sp.lk - sp.lq;
    int prefix = 0;
    if (p.prefix) prefix = (int)clamp64(p.prefix[sp.seq], 0, sp.lk);
    auto limit = [&](int i) { return p.causal ? max(min(max(i + shift + 1, prefix), sp.lk), 0) : sp.lk; };
    const int row0 = sp.tile * kBM + wave * 32, row = row0 + lane % 32;
    const int wg_limit = limit(min(sp.tile * kBM + kBM, sp.lq) - 1);
    const int ntiles = (wg_limit + KT - 1) / KT;
    const int my_limit = row < sp.lq ? limit(row) : 0;
    const int wave_most = row0 < sp.lq ? limit(min(row0 + 32, sp.lq) - 1) : 0;
    const int wave_least = limit(row0);

    const T* kg = static_cast<const T*>(p.k) + sp.k0 * p.k_stride + (int64_t)kvh * D;
    const T* vg = static_cast<const T*>(p.v) + sp.k0 * p.v_stride + (int64_t)kvh * D;
    const int64_t mine = (sp.q0 + min(row, sp.lq - 1)) * p.H + head;  // this lane's (query, head)

    Frag qf[NT], gf[NT];
    float delta = 0.f;
    {
        const T* qg = static_cast<const T*>(p.q) + (sp.q0 + min(row, sp.lq - 1)) * p.q_stride + (int64_t)head * D;
        const T* gg = static_cast<const T*>(p.dy) + mine * D;
        const T* yg = static_cast<const T*>(p.y) + mine * D;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int at = (2 * t + half) * O::kE;
            qf[t] = __builtin_bit_cast(Frag, ld16(qg + at));
            gf[t] = __builtin_bit_cast(Frag, ld16(gg + at));
            const Frag yf = __builtin_bit_cast(Frag, ld16(yg + at));
#pragma unroll
            for (int e = 0; e < O::kE; ++e) delta += (float)gf[t][e] * (float)yf[e];
        }
    }
    delta += other_half(delta);
    float lse2 = p.lse[mine] * kLog2e;
    // a row that sees nothing, and the tile's rows past the last query: all their weights are zero
    if (lse2 == -INFINITY || row >= sp.lq) lse2 = INFINITY;

    Score sc;
    sc.init(p.scale, p.cap, CAP, sizeof(T) == 4);
    float slope2 = 0.f;
    if constexpr (BIAS == kBiasSlopes) slope2 = p.slopes[head] * kLog2e;
    const int md = p.bk.max_distance, reach = 2 * md + 1;
    float* lut = extra;
    float* sums = extra + reach + wave * reach;                                 // by relative position
    float* block = extra + (1 + kWaves) * reach + wave * kDiagBlock;            // dS [key][query]
    float* far = extra + (1 + kWaves) * reach + kWaves * kDiagBlock;            // [2][kWaves]
    if constexpr (BIAS == kBiasBuckets) {
        fill_bias(lut, p, head);
        if (grad)
            for (int i = lane; i < reach; i += kWave) sums[i] = 0.f;
    }
    float far_lo = 0.f, far_hi = 0.f;
    const int qpos = row + shift;

    f32x16 acc[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) acc[d] = f32x16{};

    uint4 kb[L::kLoads], vb[L::kLoads];
    for (int pass = grad ? 0 : 1; pass < 2; ++pass) {
        float exact = 0.f;
        if (ntiles > 0) {
            L::load(kb, kg, p.k_stride, 0, sp.lk - 1);
            L::load(vb, vg, p.v_stride, 0, sp.lk - 1);
            L::store(ks[0], kb);
            L::store(vs[0], vb);
        }
        __syncthreads();
        for (int t = 0; t < ntiles; ++t) {
            const int k0 = t * KT;
            if (t + 1 < ntiles) {
                L::load(kb, kg, p.k_stride, k0 + KT, sp.lk - 1);
                L::load(vb, vg, p.v_stride, k0 + KT, sp.lk - 1);
            }
            const T* kt = ks[t & 1];
            const T* vt = vs[t & 1];
            if (k0 < wave_most) {
#pragma unroll
                for (int n = 0; n < NS; ++n) {
                    f32x16 s{}, dp{};
#pragma unroll
                    for (int i = 0; i < NT; ++i) s = O::mma(L::rows(kt, 32 * n, i, lane), qf[i], s);
#pragma unroll
                    for (int i = 0; i < NT; ++i) dp = O::mma(L::rows(vt, 32 * n, i, lane), gf[i], dp);
                    const int kn = k0 + 32 * n, rel0 = kn + 4 * half - qpos;
                    f32x16 slope;  // derivative of the cap
                    if constexpr (CAP) {
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            const float u = sc.template tanh_of<T>(s[r]);
                            s[r] = sc.c2 * u;
                            slope[r] = 1.f - u * u;
                        }
                    }
                    const float a = CAP ? 1.f : sc.a;
                    bool near = false;
                    if constexpr (BIAS == kBiasNone) {
                        if constexpr (!CAP) s *= a;
                    } else if constexpr (BIAS == kBiasSlopes) {
                        const float rel = (float)rel0;
#pragma unroll
                        for (int r = 0; r < 16; ++r) s[r] = s[r] * a - slope2 * fabsf(rel + (float)acc_row(r));
                    } else {
                        const int lowest = kn - (row0 + 31 + shift), highest = kn + 31 - (row0 + shift);
                        near = highest > -md && lowest < md;
                        if (!near) {
                            const float b = lut[highest <= -md ? 0 : 2 * md];
#pragma unroll
                            for (int r = 0; r < 16; ++r) s[r] = s[r] * a + b;
                        } else {
#pragma unroll
                            for (int r = 0; r < 16; ++r) s[r] = s[r] * a + lut[min(max(rel0 + acc_row(r), -md), md) + md];
                        }
                    }
                    if (kn + 32 > wave_least) {
                        const int left = my_limit - kn - 4 * half;
#pragma unroll
                        for (int r = 0; r < 16; ++r) s[r] = acc_row(r) < left ? s[r] : -INFINITY;
                    }
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = exp2_hw(s[r] - lse2);
                    if (pass == 0) {
#pragma unroll
                        for (int r = 0; r < 16; ++r) exact += s[r] * dp[r];
                        continue;
                    }
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] *= dp[r] - delta;
                    if constexpr (BIAS == kBiasBuckets) {
                        if (grad && !near) {
                            float add = 0.f;
#pragma unroll
                            for (int r = 0; r < 16; ++r) add += s[r];
                            if (kn < row0 + shift) far_lo += add; else far_hi += add;
                        } else if (grad) {
                            // sums along the diagonals of 16 keys x 32 queries: lane j takes relative
                            // position base + j, from the corner key 0, query 31 on
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
#pragma unroll
                                for (int r = 0; r < 8; ++r) block[(acc_row(r) + 4 * half) * kDiagStride + lane % 32] = s[8 * b + r];
                                __builtin_amdgcn_wave_barrier();
                                const int off = lane - 31, rel = kn + 16 * b - (row0 + shift) + off;
                                float add = 0.f;
                                for (int key = max(off, 0); key < kDiagRows && key - off < 32; ++key)
                                    add += block[key * kDiagStride + key - off];
                                if (lane < 31 + kDiagRows) {
                                    if (rel <= -md) far_lo += add;
                                    else if (rel >= md) far_hi += add;
                                    else sums[rel + md] += add;
                                }
                                __builtin_amdgcn_wave_barrier();
                            }
                        }
                    }
                    if constexpr (CAP) s *= slope;
#pragma unroll
                    for (int kk = 0; kk < PK; ++kk) {
                        const Frag sf = O::pack(s, kk);
#pragma unroll
                        for (int d = 0; d < DT; ++d) acc[d] = O::mma(L::cols(kt, 32 * n, kk, 32 * d, lane), sf, acc[d]);
                    }
                }
            }
            if (t + 1 < ntiles) {
                L::store(ks[(t + 1) & 1], kb);
                L::store(vs[(t + 1) & 1], vb);
            }
            lds_barrier();
        }
        if (pass == 0) delta = exact + other_half(exact);
    }

    if (row < sp.lq) {
        if (half == 0) p.delta[mine] = delta;
        T* out = static_cast<T*>(p.dq) + mine * D;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            acc[d] *= p.scale;
#pragma unroll
            for (int r = 0; r < 16; r += 4)
                store4(out + 32 * d + 2 * r + 4 * half, acc[d][r], acc[d][r + 1], acc[d][r + 2], acc[d][r + 3]);
        }
    }
    if constexpr (BIAS == kBiasBuckets) {
        if (!grad) return;
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) {
            far_lo += __shfl_xor(far_lo, off, kWave);
            far_hi += __shfl_xor(far_hi, off, kWave);
        }
        if (lane == 0) {
            far[wave] = far_lo;
            far[kWaves + wave] = far_hi;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < p.bk.total; i += kThreads) {
            float v = 0.f;
            for (int w = 0; w < kWaves; ++w) {
                v += fold_bucket(p.bk, extra + reach + w * reach, i);
                if (i == p.bk.nborders) v += far[w];  // the last bucket of the first direction
                if (i == (p.bk.both ? p.bk.total - 1 : 0)) v += far[kWaves + w];
            }
            part[i] = v;
        }
    }
}

// dtable[b, h]: the query tiles' sums, in order.
__global__ void __launch_bounds__(kThreads) attn_dtable_kernel(AttnParams p) {
    __shared__ double sums[kThreads];
    const int nb = p.bk.total, head = blockIdx.x, groups = kThreads / nb;
    const int b = threadIdx.x % nb, g = threadIdx.x / nb;
    double v = 0.0;
    if (g < groups)
        for (int s = g; s < p.q_slots; s += groups) v += (double)p.table_part[((int64_t)s * p.H + head) * nb + b];
    sums[threadIdx.x] = v;
    __syncthreads();
    if (g == 0) {
        for (int i = 1; i < groups; ++i) v += sums[i * nb + b];
        p.dtable[(int64_t)b * p.H + head] = (float)v;
    }
}

template <typename T, int D, bool CAP, int BIAS>
__global__ void __launch_bounds__(kThreads, sizeof(T) * D >= 256 ? 1 : 2) attn_dkv_kernel(AttnParams p) {
    using O = Op<T>;
    using L = Tile<T, D>;
    using Frag = typename O::Frag;
    constexpr int QT = O::kKT, NS = QT / 32, NT = D / O::kK, DT = D / 32, PK = 32 / O::kK;
    __shared__ __attribute__((aligned(16))) T qs[2][L::kElems];
    __shared__ __attribute__((aligned(16))) T gs[2][L::kElems];
    __shared__ __attribute__((aligned(16))) float stat[2][2][QT];  // [buffer][lse in log2 units, D][query]
    extern __shared__ float extra[];
    float* lut = extra;

    int slot, kvh;
    work_item(blockIdx.x, p.k_slots, p.Hk, slot, kvh);
    slot = p.k_slots - 1 - slot;  // under a causal mask the first keys are seen by the most queries
    const Span sp = find_span(p, slot, true);
    if (sp.tile < 0) return;
    const int group = p.H / p.Hk;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, half = lane / 32;
    const int shift = sp.lk - sp.lq;
    int prefix = 0;
    if (p.prefix) prefix = (int)clamp64(p.prefix[sp.seq], 0, sp.lk);

    // queries [first(j), lq) see key j
    auto first = [&](int j) { return !p.causal || j < prefix ? 0 : max(j - shift, 0); };
    const int row0 = sp.tile * kBM + wave * 32, key = row0 + lane % 32;
    const int t0 = first(sp.tile * kBM) / QT, t1 = (sp.lq + QT - 1) / QT;
    const int my_first = key < sp.lk ? first(key) : sp.lq;
    const int wave_least = row0 < sp.lk ? first(row0) : sp.lq;  // the earliest query that any key of the wave meets
    const int wave_most = row0 + 32 <= sp.lk ? first(row0 + 31) : sp.lq;  // from here on every key meets every query
    const int per_head = max(t1 - t0, 0), ntiles = per_head * group;

    const int64_t krow = sp.k0 + min(key, sp.lk - 1);
    Frag kf[NT], vf[NT];
    {
        const T* kg = static_cast<const T*>(p.k) + krow * p.k_stride + (int64_t)kvh * D;
        const T* vg = static_cast<const T*>(p.v) + krow * p.v_stride + (int64_t)kvh * D;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            kf[t] = __builtin_bit_cast(Frag, ld16(kg + (2 * t + half) * O::kE));
            vf[t] = __builtin_bit_cast(Frag, ld16(vg + (2 * t + half) * O::kE));
        }
    }
    Score sc;
    sc.init(p.scale, p.cap, CAP, sizeof(T) == 4);
    const int md = p.bk.max_distance;

    f32x16 dk[DT], dv[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) dk[d] = dv[d] = f32x16{};

    uint4 qb[L::kLoads], gb[L::kLoads];
    float sb = 0.f;  // threads 0 .. QT - 1: lse, the next QT: D
    auto fetch = [&](int it) {
        const int head = kvh * group + it / per_head, first_row = (t0 + it % per_head) * QT;
        L::load(qb, static_cast<const T*>(p.q) + sp.q0 * p.q_stride + (int64_t)head * D, p.q_stride, first_row, sp.lq - 1);
        L::load(gb, static_cast<const T*>(p.dy) + (sp.q0 * p.H + head) * D, (int64_t)p.H * D, first_row, sp.lq - 1);
        if (threadIdx.x < 2 * QT) {
            const int64_t at = (sp.q0 + min(first_row + (int)threadIdx.x % QT, sp.lq - 1)) * p.H + head;
            if (threadIdx.x < QT) {
                sb = p.lse[at] * kLog2e;
                if (sb == -INFINITY) sb = INFINITY;
            } else {
                sb = p.delta[at];
            }
        }
    };
    auto put = [&](int buf) {
        L::store(qs[buf], qb);
        L::store(gs[buf], gb);
        if (threadIdx.x < 2 * QT) stat[buf][threadIdx.x / QT][threadIdx.x % QT] = sb;
    };
    if (ntiles > 0) {
        fetch(0);
        put(0);
    }

    for (int it = 0; it < ntiles; ++it) {
        const int head = kvh * group + it / per_head, q0 = (t0 + it % per_head) * QT;
        if constexpr (BIAS == kBiasBuckets) {
            if (it % per_head == 0) {  // (the barrier at the end of the last round: nobody reads the old one)
                fill_bias(lut, p, head);
            }
        }
        if (it == 0 || (BIAS == kBiasBuckets && it % per_head == 0)) __syncthreads();
        float slope2 = 0.f;
        if constexpr (BIAS == kBiasSlopes) slope2 = p.slopes[head] * kLog2e;
        if (it + 1 < ntiles) fetch(it + 1);
        const T* qt = qs[it & 1];
        const T* gt = gs[it & 1];
        if (q0 + QT > wave_least) {
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                f32x16 s{}, dp{};
#pragma unroll
                for (int i = 0; i < NT; ++i) s = O::mma(L::rows(qt, 32 * n, i, lane), kf[i], s);
#pragma unroll
                for (int i = 0; i < NT; ++i) dp = O::mma(L::rows(gt, 32 * n, i, lane), vf[i], dp);
                const int qn = q0 + 32 * n;
                const int rel0 = key - (qn + shift + 4 * half);  // of register 0; later queries are further on
                f32x16 slope;
                if constexpr (CAP) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const float u = sc.template tanh_of<T>(s[r]);
                        s[r] = sc.c2 * u;
                        slope[r] = 1.f - u * u;
                    }
                }
                const float a = CAP ? 1.f : sc.a;
                if constexpr (BIAS == kBiasNone) {
                    if constexpr (!CAP) s *= a;
                } else if constexpr (BIAS == kBiasSlopes) {
                    const float rel = (float)rel0;
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = s[r] * a - slope2 * fabsf(rel - (float)acc_row(r));
                } else {
                    const int lowest = row0 - (qn + 31 + shift), highest = row0 + 31 - (qn + shift);
                    if (highest <= -md || lowest >= md) {
                        const float b = lut[highest <= -md ? 0 : 2 * md];
#pragma unroll
                        for (int r = 0; r < 16; ++r) s[r] = s[r] * a + b;
                    } else {
#pragma unroll
                        for (int r = 0; r < 16; ++r) s[r] = s[r] * a + lut[min(max(rel0 - acc_row(r), -md), md) + md];
                    }
                }
                if (qn < wave_most || qn + 32 > sp.lq) {
                    const int lo = my_first - qn - 4 * half, hi = sp.lq - qn - 4 * half;
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = acc_row(r) >= lo && acc_row(r) < hi ? s[r] : -INFINITY;
                }
                const float* ls = &stat[it & 1][0][32 * n + 4 * half];
                const float* de = &stat[it & 1][1][32 * n + 4 * half];
#pragma unroll
                for (int r = 0; r < 16; r += 4) {
                    const f32x4 lv = as_f32x4(ld16(ls + acc_row(r))), dl = as_f32x4(ld16(de + acc_row(r)));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[r + e] = exp2_hw(s[r + e] - lv[e]);
                        dp[r + e] = s[r + e] * (dp[r + e] - dl[e]);
                    }
                }
                if constexpr (CAP) dp *= slope;
#pragma unroll
                for (int kk = 0; kk < PK; ++kk) {
                    const Frag pf = O::pack(s, kk), sf = O::pack(dp, kk);
#pragma unroll
                    for (int d = 0; d < DT; ++d) {
                        dv[d] = O::mma(L::cols(gt, 32 * n, kk, 32 * d, lane), pf, dv[d]);
                        dk[d] = O::mma(L::cols(qt, 32 * n, kk, 32 * d, lane), sf, dk[d]);
                    }
                }
            }
        }
        if (it + 1 < ntiles) put((it + 1) & 1);
        lds_barrier();
    }

    if (key >= sp.lk) return;
    T* dkg = static_cast<T*>(p.dk) + ((sp.k0 + key) * p.Hk + kvh) * D;
    T* dvg = static_cast<T*>(p.dv) + ((sp.k0 + key) * p.Hk + kvh) * D;
#pragma unroll
    for (int d = 0; d < DT; ++d) {
        dk[d] *= p.scale;
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
            store4(dkg + 32 * d + 2 * r + 4 * half, dk[d][r], dk[d][r + 1], dk[d][r + 2], dk[d][r + 3]);
            store4(dvg + 32 * d + 2 * r + 4 * half, dv[d][r], dv[d][r + 1], dv[d][r + 2], dv[d][r + 3]);
        }
    }
}

template <typename T, int D, bool CAP, int BIAS>
int launch_bwd(const AttnParams& p, hipStream_t stream) {
    const int64_t q_grid = (int64_t)p.q_slots * p.H, k_grid = (int64_t)p.k_slots * p.Hk;
    const size_t q_lds = 4 * (size_t)bias_floats(BIAS, p.bk.max_distance, p.dtable != nullptr);
    const size_t k_lds = 4 * (size_t)bias_floats(BIAS, p.bk.max_distance, false);
    if (BIAS == kBiasBuckets) {
        if (hipFuncSetAttribute(reinterpret_cast<const void*>(&attn_dq_kernel<T, D, CAP, BIAS>),
                                hipFuncAttributeMaxDynamicSharedMemorySize, (int)q_lds) != hipSuccess ||
            hipFuncSetAttribute(reinterpret_cast<const void*>(&attn_dkv_kernel<T, D, CAP, BIAS>),
                                hipFuncAttributeMaxDynamicSharedMemorySize, (int)k_lds) != hipSuccess)
            return -1;
    }
    if (q_grid > 0) {
        hipLaunchKernelGGL((attn_dq_kernel<T, D, CAP, BIAS>), dim3((unsigned)q_grid), dim3(kThreads), q_lds, stream, p);
        if (hipGetLastError() != hipSuccess) return -1;
    }
    if (p.dtable) {
        hipLaunchKernelGGL(attn_dtable_kernel, dim3((unsigned)p.H), dim3(kThreads), 0, stream, p);
        if (hipGetLastError() != hipSuccess) return -1;
    }
    if (k_grid > 0) {
        hipLaunchKernelGGL((attn_dkv_kernel<T, D, CAP, BIAS>), dim3((unsigned)k_grid), dim3(kThreads), k_lds, stream, p);
        if (hipGetLastError() != hipSuccess) return -1;
    }
    return 0;
}
template <typename T, int D, bool CAP>
int launch_bwd(const AttnParams& p, int bias, hipStream_t stream) {
    switch (bias) {
        case kBiasNone: return launch_bwd<T, D, CAP, kBiasNone>(p, stream);
        case kBiasSlopes: return launch_bwd<T, D, CAP, kBiasSlopes>(p, stream);
        default: return launch_bwd<T, D, CAP, kBiasBuckets>(p, stream);
    }
}
template <typename T>
int launch_bwd(const AttnParams& p, int D, int bias, hipStream_t stream) {
    const bool cap = p.cap > 0.f;
    switch (D) {
        case 32: return cap ? launch_bwd<T, 32, true>(p, bias, stream) : launch_bwd<T, 32, false>(p, bias, stream);
        case 64: return cap ? launch_bwd<T, 64, true>(p, bias, stream) : launch_bwd<T, 64, false>(p, bias, stream);
        case 128: return cap ? launch_bwd<T, 128, true>(p, bias, stream) : launch_bwd<T, 128, false>(p, bias, stream);
        default: return -2;
    }
}

}  // namespace
}  // namespace attn

int launch_attn_backward(const AttnParams& in, int dtype, int D, int bias, hipStream_t stream) {
    AttnParams p = in;
    p.q_slots = (int)attn::slots_of(p.cu_q, p.total_q, p.nseq);
    p.k_slots = (int)attn::slots_of(p.cu_k, p.total_k, p.nseq);
    return dtype == 1 ? attn::launch_bwd<__bf16>(p, D, bias, stream) : attn::launch_bwd<float>(p, D, bias, stream);
}

}  // namespace ssd
