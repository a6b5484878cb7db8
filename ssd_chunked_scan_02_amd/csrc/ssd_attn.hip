// Attention over a packed batch of documents, forward, gfx950:
//     s_ij = scale q_i.k_j, capped to c tanh(s / c), plus a bias by distance;  p = softmax over the
//     visible j;  y_i = sum_j p_ij v_j;  lse_i = log sum_j exp s_ij.
//
// One pass over the keys with a running maximum m and sum l (in log2 units): a workgroup of four waves
// owns 128 query rows (of one head, or of all heads of a group) of a document, 32 a wave, and streams
// 64-key tiles (32 in fp32) through LDS, double buffered, the next tile on its way to LDS while the present
// one is used.  A wave forms
// S^T = K Q^T (queries in lanes), so m and l are one number a lane, and P^T in its accumulator layout is
// the operand of O^T += V^T P^T (ssd_attn_common.h).  O is rescaled only when a row's maximum has grown by
// more than 2^8: weights are relative to m, so a late m costs no accuracy.  In bf16 a weight is rounded for the
// product with V; y is divided by the sum of the rounded weights, so that what their rounding has in
// common drops out (a row of one key gives that value exactly, as the backward pass needs: it forms
// dy.y - dy.v), and lse comes from the sum of the unrounded ones.  With too few rows to fill
// the chip the waves split the keys instead (SPLIT).
//
// A row's y depends on the keys that it sees, whatever lies in the others of its tile: a weight of zero does not keep
// an infinity or NaN of V out of a product (the copies of the last key that fill its tile have that weight, too), so
// where one has come up the workgroup does its tiles again with those values taken out (attn_fwd_rows<CAREFUL>).  A row
// sees the keys before its limit, so that the first key with a NaN, an infinity and a negative infinity in a column say
// what that column of the row is.  (The vote costs 0.3 us of the 11.5 of 256 tokens of one head, and nothing that 2 ms of
// a long prompt show.)
//
// Measured: 16384 tokens, 32/4 heads of 128, causal, bf16: 2.10 to 2.25 ms from box to box, 0.98 to 1.04 PFLOP/s, 81 to 86% of
// what an 8192^3 matrix product reaches; MFMA is busy for 52% of its cycles and VALU for 53%, in turns.  8 x 2048 tokens,
// 24 heads of 64, capped: 182 to 200 us, 530 TFLOP/s, bound by VALU (84% of the cycles in which a CU has a wave, which are
// 82%): a score costs 11 instructions, one of them an exponential of four issue slots, against 4 MFMA cycles a lane.
// The tile: 32 queries a wave and 64 keys read LDS at half its rate when MFMA is full and leave registers for two
// (128-wide heads) or three waves a SIMD; 32 keys at a time measured 2.30 against 2.17 ms at 128 wide.
#include "ssd_attn_common.h"

namespace ssd {
namespace attn {
namespace {

constexpr float kLazy = 8.f;  // log2 growth of a maximum that is let pass without a rescale
// Scores capped to at most 2^80 need no maximum at all: weights in [2^-80, 2^80] and their sums stay inside fp32 (and
// bf16, which has its range).  Where their products with V may not (a sum is infinite, or a row's weights come to less
// than 2^-32), the workgroup does its tiles again, with a maximum for those rows (attn_fwd_rows<CAREFUL>, `track`).
constexpr float kNoMaxNeeded = 80.f, kFewWeights = 0x1p-32f;
enum Cap { kCapNone = 0, kCapped = 1, kCapBounds = 2 };  // kCapBounds: without a bias, by a cap that needs no maximum

// LDS, in arrays of their own: a load on its way to one is not waited for at another.
template <typename T, int D, bool SPLIT> struct FwdShared {
    static constexpr int KT = SPLIT ? 32 : Op<T>::kKT, ELEMS = (SPLIT ? kWaves : 1) * KT * D;
    static constexpr bool DOUBLE = !SPLIT || ELEMS * sizeof(T) <= 32768;  // (two buffers of split fp32 tiles of 128 would not fit)
    T *k_a, *v_a, *k_b, *v_b;
    float* lut;
    float (*stat)[SPLIT ? kWaves * 32 : 1];  // by row: m, l, weight of a wave's share, sum of rounded weights
    int (*first)[D];                         // CAREFUL, by column of V: first key with a NaN, an infinity, a negative one
};

// The rows of workgroup `block`; CAREFUL: what is infinite or NaN in V counts for the rows that see it, and for no others.
// Returns whether something infinite or NaN came up, or a row needs the maximum that it was done without;
// CAREFUL: the latter, of this lane's row (SPLIT: this wave's share of it).
template <typename T, int D, int CAPPED, int BIAS, bool SPLIT, bool CAREFUL>
__device__ __forceinline__ bool attn_fwd_rows(const AttnParams& p, const FwdShared<T, D, SPLIT>& lds, uint32_t block, int tid, bool track) {
    using O = Op<T>;
    using L = Tile<T, D>;
    using Frag = typename O::Frag;
    constexpr int OWN = kOwn<SPLIT>, KT = SPLIT ? 32 : O::kKT, NS = KT / 32, NT = D / O::kK, DT = D / 32, PK = 32 / O::kK;
    constexpr bool DOUBLE = FwdShared<T, D, SPLIT>::DOUBLE;
    constexpr bool CAP = CAPPED != kCapNone, NO_MAX = CAPPED == kCapBounds;
    constexpr bool RAW = !CAP && BIAS == kBiasNone;  // scores stay raw products until the exponential
    constexpr bool ROUNDED = sizeof(T) == 2;  // weights lose bits on their way to V
    T *const k_a = lds.k_a, *const v_a = lds.v_a, *const k_b = lds.k_b, *const v_b = lds.v_b;
    const auto stat = lds.stat;
    const auto first = lds.first;

    int slot, unit;
    work_item(block, p.q_slots, (uint32_t)p.H / (uint32_t)p.pack, slot, unit);
    const Span sp = find_span(p, slot, OWN, false);
    if (sp.tile < 0) return false;
    const int head0 = unit * p.pack, kvh = (int)((uint32_t)head0 / ((uint32_t)p.H / (uint32_t)p.Hk));
    const int lane = tid % kWave, half = lane / 32;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int shift = sp.lk - sp.lq;  // position of query 0 on the key axis
    int prefix = 0;
    if (p.prefix) prefix = (int)clamp64(p.prefix[sp.seq], 0, sp.lk);

    // keys [0, limit(i)) are visible to query i
    auto limit = [&](int i) { return p.causal ? max(min(max(i + shift + 1, prefix), sp.lk), 0) : sp.lk; };
    const int row0 = sp.tile * OWN + (SPLIT ? 0 : wave * 32), row = row0 + lane % 32;
    auto query_of = [&](int r) { return (int)((uint32_t)r / (uint32_t)p.pack); };
    const int mine = query_of(min(row, sp.rows - 1)), head = head0 + min(row, sp.rows - 1) - mine * p.pack;
    const int wg_limit = limit(query_of(min(sp.tile * OWN + OWN, sp.rows) - 1));
    const int ntiles = (wg_limit + KT - 1) / KT;
    const int my_limit = row < sp.rows ? limit(mine) : 0;
    const int wave_most = row0 < sp.rows ? limit(query_of(min(row0 + 32, sp.rows) - 1)) : 0;  // any query of the wave
    const int wave_least = limit(query_of(row0));                                             // every query of the wave

    const T* kg = static_cast<const T*>(p.k) + sp.k0 * p.k_stride + (int64_t)kvh * D;
    const T* vg = static_cast<const T*>(p.v) + sp.k0 * p.v_stride + (int64_t)kvh * D;
    Feed<T, D, KT, SPLIT ? kWave : kThreads> kf, vf;
    kf.init(p.k_stride);
    vf.init(p.v_stride);
    const int at = SPLIT ? wave * KT * D : 0;
    T *ka = k_a + at, *va = v_a + at, *kb = k_b + (DOUBLE ? at : 0), *vb = v_b + (DOUBLE ? at : 0);
    auto fetch = [&](T* ks, T* vs, int t) {
        kf.load(ks, kg, t * KT, sp.lk - t * KT);
        vf.load(vs, vg, t * KT, sp.lk - t * KT);
    };
    const int t0 = SPLIT ? wave : 0, dt = SPLIT ? kWaves : 1;
    if (t0 < ntiles) fetch(ka, va, t0);

    Frag qf[NT];
    {
        const T* qg = static_cast<const T*>(p.q) + (sp.q0 + mine) * p.q_stride + (int64_t)head * D;
#pragma unroll
        for (int t = 0; t < NT; ++t) qf[t] = signed_frag<T>(qg + (2 * t + half) * O::kE, p.scale);
    }
    Score sc;
    sc.init<T>(fabsf(p.scale), p.cap, CAP);
    float slope2 = 0.f;
    if constexpr (BIAS == kBiasSlopes) slope2 = p.slopes[head] * kLog2e;
    if constexpr (BIAS == kBiasBuckets) fill_bias(lds.lut, p, head);

    f32x16 o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = f32x16{};
    float m = NO_MAX && !(CAREFUL && track) ? 0.f : kNoMax, l = 0.f, lr = 0.f;  // this lane half's share of the weights, and of the rounded ones
    const int qpos = mine + shift;
    if constexpr (CAREFUL) {
        for (int i = tid; i < 3 * D; i += kThreads) first[0][i] = INT_MAX;
        __syncthreads();
    }
    // a column of y from its sum over what is finite in V
    auto with_rest = [&](float x, int column, int see) {
        const bool nan = first[0][column] < see, up = first[1][column] < see, down = first[2][column] < see;
        return nan || (up && down) ? NAN : x != x ? x : up ? INFINITY : down ? -INFINITY : x;
    };

    auto meet = [&]() {
        if constexpr (SPLIT) __builtin_amdgcn_wave_barrier(); else lds_barrier();
    };
    // what was on its way to LDS (the values of tile t: to v) is there, and (SPLIT: this wave's) reads are over
    auto settle = [&](T* v, int t) {
        __builtin_amdgcn_s_waitcnt(SPLIT ? kAllDone : kLoadsDone);
        meet();
        if (CAREFUL && v) {
            vf.clean(v, t * KT, first);
            __builtin_amdgcn_s_waitcnt(kAllDone);
            meet();
        }
    };
    const typename L::Lanes z(lane);
    auto step = [&](const T* kt, const T* vt, T* kn, T* vn, int t) {
        const int k0 = t * KT;
        if (DOUBLE && t + dt < ntiles) fetch(kn, vn, t + dt);
        if (k0 < wave_most) {
            f32x16 s[NS];
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                s[n] = f32x16{};
#pragma unroll
                for (int i = 0; i < NT; ++i) s[n] = O::mma(L::rows(kt, 32 * n, i, z), qf[i], s[n]);
            }
            if constexpr (CAP) sc.template capped<T>(s);
            add_bias<BIAS, 1>(s, CAP ? 1.f : sc.a, slope2, lds.lut, p.bk.max_distance, k0 + 4 * half - qpos,
                              k0 - (row0 + 31 + shift), k0 + KT - 1 - (row0 + shift));
            if (k0 + KT > wave_least) {
                const int left = my_limit - k0 - 4 * half;
#pragma unroll
                for (int n = 0; n < NS; ++n)
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[n][r] = 32 * n + acc_row(r) < left ? s[n][r] : -INFINITY;
            }
            if constexpr (!NO_MAX || CAREFUL) {
                float mx = s[0][0];
#pragma unroll
                for (int n = 0; n < NS; ++n)
#pragma unroll
                    for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[n][r]);
                mx = fmaxf(mx, other_half(mx));
                if constexpr (RAW) mx *= sc.a;
                const bool grown = mx > m + kLazy && (!NO_MAX || track);
                if (__any(grown)) {
                    // (each row by its own growth, so that its weights' rounding does not depend on the others)
                    const float next = grown ? mx : m, keep = exp2_hw(m - next);
                    m = next;
                    l *= keep;
                    lr *= keep;
#pragma unroll
                    for (int d = 0; d < DT; ++d) o[d] *= keep;
                }
            }
            float add = 0.f;
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    s[n][r] = exp2_hw(RAW ? __builtin_fmaf(s[n][r], sc.a, -m) : NO_MAX && !CAREFUL ? s[n][r] : s[n][r] - m);
                    add += s[n][r];
                }
            l += add;
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int kk = 0; kk < PK; ++kk) {
                    const Frag pf = O::pack(s[n], kk);
                    if constexpr (ROUNDED) lr = sum_of(pf, lr);
#pragma unroll
                    for (int d = 0; d < DT; ++d) o[d] = O::mma(L::cols(vt, 32 * n, kk, 32 * d, z), pf, o[d]);
                }
        }
        settle(DOUBLE && t + dt < ntiles ? vn : nullptr, t + dt);
        if (!DOUBLE && t + dt < ntiles) {
            fetch(kn, vn, t + dt);
            settle(vn, t + dt);
        }
    };
    if constexpr (SPLIT && BIAS == kBiasBuckets) __syncthreads();  // (the bias is everybody's)
    settle(t0 < ntiles ? va : nullptr, t0);
    for (int t = t0; t < ntiles; t += 2 * dt) {
        step(ka, va, DOUBLE ? kb : ka, DOUBLE ? vb : va, t);
        if (t + dt < ntiles) step(DOUBLE ? kb : ka, DOUBLE ? vb : va, ka, va, t + dt);
    }

    l += other_half(l);
    if constexpr (ROUNDED) lr += other_half(lr); else lr = l;
    float bad = 0.f;
    if constexpr (!CAREFUL || NO_MAX) {
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r) bad = __builtin_fmaf(o[d][r], 0.f, bad);
        if (NO_MAX && l > 0.f && l < kFewWeights) bad = 1.f;
        if constexpr (CAREFUL) bad += other_half(bad);  // (a row's two lanes keep one maximum)
    }
    if constexpr (SPLIT) {
        if (half == 0) {
            stat[0][32 * wave + lane] = m;
            stat[1][32 * wave + lane] = l;
            stat[3][32 * wave + lane] = lr;
        }
        __syncthreads();  // (nobody reads a tile any more)
        Join<T, D>::keep(k_a, v_a, o, lane, wave);
        if (tid < 32) {
            float top = kNoMax, sum = 0.f, rounded = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) top = fmaxf(top, stat[0][32 * w + lane]);
            float f[kWaves];
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                f[w] = exp2_hw(stat[0][32 * w + lane] - top);
                sum += f[w] * stat[1][32 * w + lane];
                rounded += f[w] * stat[3][32 * w + lane];
            }
            const float inv = rounded > 0.f ? 1.f / rounded : (rounded == 0.f ? 0.f : rounded);
#pragma unroll
            for (int w = 0; w < kWaves; ++w) stat[2][32 * w + lane] = f[w] * inv;
            if (row < sp.rows && p.lse)
                p.lse[(sp.q0 + mine) * p.H + head] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * kLn2;
        }
        __syncthreads();
        for (int i = tid; i < 32 * (D / 4); i += kThreads) {
            const int r = i / (D / 4), d4 = i % (D / 4);
            if (row0 + r >= sp.rows) break;
            f32x4 v = Join<T, D>::sum(k_a, v_a, r, d4, stat[2]);
            const int q = query_of(row0 + r);
            if constexpr (CAREFUL) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = with_rest(v[e], 4 * d4 + e, limit(q));
            }
            store4(static_cast<T*>(p.y) + ((sp.q0 + q) * p.H + head0 + row0 + r - q * p.pack) * D + 4 * d4, v[0], v[1], v[2], v[3]);
        }
    } else if (row < sp.rows) {
        // (the store exchanges words between a row's two lanes, which are in or out together)
        float inv = lr > 0.f ? 1.f / lr : (lr == 0.f ? 0.f : lr);  // (an empty row is zero; a NaN stays one)
        if constexpr (CAREFUL) {
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[d][r] = with_rest(o[d][r] * inv, 32 * d + acc_row(r) + 4 * half, my_limit);
            inv = 1.f;
        }
        T* yg = static_cast<T*>(p.y) + ((sp.q0 + mine) * p.H + head) * D;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int r = 0; r < 16; r += 8) store_rows(yg + 32 * d, o[d], r, half, inv);
        if (p.lse && half == 0) p.lse[(sp.q0 + mine) * p.H + head] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
    }

    return bad != 0.f && !(CAREFUL && track);
}

// Waves a SIMD.  Capped scores without a maximum: as many as the first pass's registers leave room for; the second pass,
// with a maximum, has to do with those (left to itself it takes a wave from the first at 32- and 64-wide heads).
template <int ROW, int D, int CAPPED, bool SPLIT>
constexpr int kForwardWaves = CAPPED != kCapBounds ? (SPLIT || ROW >= 512 ? 1 : 2)
                              : SPLIT              ? (ROW <= 64 ? 3 : ROW <= 128 ? 2 : 1)
                                                   : (D == 32 ? 4 : D == 64 ? 3 : ROW <= 256 ? 2 : 1);

template <typename T, int D, int CAPPED, int BIAS, bool SPLIT>
__global__ void __launch_bounds__(kThreads, (kForwardWaves<(int)sizeof(T) * D, D, CAPPED, SPLIT>)) attn_fwd_kernel(AttnParams p) {
    using S = FwdShared<T, D, SPLIT>;
    __shared__ __attribute__((aligned(16))) T k_a[S::ELEMS];
    __shared__ __attribute__((aligned(16))) T v_a[S::ELEMS];
    __shared__ __attribute__((aligned(16))) T k_b[S::DOUBLE ? S::ELEMS : 8];
    __shared__ __attribute__((aligned(16))) T v_b[S::DOUBLE ? S::ELEMS : 8];
    __shared__ float lut[BIAS == kBiasBuckets ? 2 * kMaxDistance + 1 : 1];
    __shared__ float stat[SPLIT ? 4 : 1][SPLIT ? kWaves * 32 : 1];
    __shared__ int first[3][D];
    const S lds{k_a, v_a, k_b, v_b, lut, stat, first};
    bool again = attn_fwd_rows<T, D, CAPPED, BIAS, SPLIT, false>(p, lds, blockIdx.x, threadIdx.x, false), track = false;
    if (!__syncthreads_or(again)) return;
    uint32_t block = blockIdx.x;
    int tid = threadIdx.x;
#pragma unroll 1
    for (int pass = 0; pass < (CAPPED == kCapBounds ? 2 : 1); ++pass) {
        asm volatile("" : "+s"(block), "+v"(tid));  // (nothing worked out for the first time is kept for this one)
        again = attn_fwd_rows<T, D, CAPPED, BIAS, SPLIT, true>(p, lds, block, tid, track);
        if (CAPPED != kCapBounds || !__syncthreads_or(again)) return;
        track = again;
    }
}

template <typename T, int D, int CAPPED, int BIAS>
int launch_fwd(AttnParams p, hipStream_t stream) {
    p.pack = query_pack(p, BIAS);
    const int units = p.H / p.pack;
    const bool split = query_slots(p, kOwn<false>) * units < attn_split_below(Tile<T, D>::RB);
    p.q_slots = (int)query_slots(p, split ? kOwn<true> : kOwn<false>);
    set_each(p, split ? kOwn<true> : kOwn<false>, 1);
    const int64_t grid = (int64_t)p.q_slots * units;
    if (grid == 0) return 0;
    if (!launchable(grid, kThreads)) return -2;
    if (split) hipLaunchKernelGGL((attn_fwd_kernel<T, D, CAPPED, BIAS, true>), dim3((unsigned)grid), dim3(kThreads), 0, stream, p);
    else hipLaunchKernelGGL((attn_fwd_kernel<T, D, CAPPED, BIAS, false>), dim3((unsigned)grid), dim3(kThreads), 0, stream, p);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}
template <typename T, int D, int CAPPED>
int launch_fwd(const AttnParams& p, int bias, hipStream_t stream) {
    switch (bias) {
        case kBiasNone:
            if (CAPPED == kCapped && p.cap * kLog2e <= kNoMaxNeeded) return launch_fwd<T, D, CAPPED ? kCapBounds : kCapNone, kBiasNone>(p, stream);
            return launch_fwd<T, D, CAPPED, kBiasNone>(p, stream);
        case kBiasSlopes: return launch_fwd<T, D, CAPPED, kBiasSlopes>(p, stream);
        default: return launch_fwd<T, D, CAPPED, kBiasBuckets>(p, stream);
    }
}
template <typename T>
int launch_fwd(const AttnParams& p, int D, int bias, hipStream_t stream) {
    const bool cap = p.cap > 0.f;
    switch (D) {
        case 32: return cap ? launch_fwd<T, 32, kCapped>(p, bias, stream) : launch_fwd<T, 32, kCapNone>(p, bias, stream);
        case 64: return cap ? launch_fwd<T, 64, kCapped>(p, bias, stream) : launch_fwd<T, 64, kCapNone>(p, bias, stream);
        case 128: return cap ? launch_fwd<T, 128, kCapped>(p, bias, stream) : launch_fwd<T, 128, kCapNone>(p, bias, stream);
        default: return -2;
    }
}

}  // namespace
}  // namespace attn

int launch_attn_forward(const AttnParams& p, int dtype, int D, int bias, hipStream_t stream) {
    return dtype == 1 ? attn::launch_fwd<__bf16>(p, D, bias, stream) : attn::launch_fwd<float>(p, D, bias, stream);
}

}  // namespace ssd
