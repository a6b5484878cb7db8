// Attention over a packed batch of documents, backward, gfx950.  With p from the forward pass's lse and
// D_i = sum_j p_ij (dy_i . v_j):
//     dS_ij = p_ij (dy_i . v_j - D_i),  dz_ij = dS_ij (1 - tanh^2),
//     dq_i = scale sum_j dz_ij k_j,  dk_j = scale sum_i dz_ij q_i,  dv_j = sum_i p_ij dy_i,
//     dtable[b] = sum of dS over the cells of bucket b.
//
// Two kernels, each owning what it sums, so that no sum is made by atomics and every run gives the
// same bits: attn_dq_kernel owns 128 query rows and streams keys (S^T, dP^T, dq^T), and leaves D for
// attn_dkv_kernel, which owns 128 keys of a key head and streams the queries of every head of its group
// (S, dP, dv^T, dk^T).  That is 7 products where sharing S and dP would need 5, and no partial
// gradients through memory.  Both keep their rows' operands and gradients in registers; the tile layout
// and operand order are the forward kernel's (ssd_attn_common.h).
//
// D is sum_d dy_id y_id to begin with, which is as exact as the given y: a bf16 y leaves it off by some e_i, and dq_i by
// scale e_i sum_j p_ij k_j.  That is little for weights spread over keys and values without a mean, but whole where a row
// has one dominating key, or keys and values a common part: dq off by 6e-2 at a mean of 2, or at a weight of 0.99 on one
// key of 2048.  The sum of a row's dS is e_i (with a bf16 dS, its own roundings' sum beside it), known after the pass, and
// with the sum of p k beside that of dS k dq is put right at the end, for one product more and registers (MEAN): 1.7e-3 to
// 2.3e-3 in all those cases (capped, where the unrounded dS is summed, 4e-3 at that mean).  The gradient of the table sums dS over whole diagonals, where e_i counts for every row: with D
// exact after the pass far cells (which share a bucket: |distance| >= max_distance) are corrected by the sum of their p,
// and the tiles near the diagonal are visited once more, for the table alone.  For 128-wide heads with a table the sum of
// p k would take a wave's room on each SIMD, and a pass over S and dP comes before instead (PASS), after which the
// diagonals are summed as dS comes up, as in fp32, whose y needs none of this.
//
// Measured in profiled runs, bf16: 8 x 2048 tokens, 24 heads of 64, capped: dq 300 to 390 us, dk and dv 322 to 428 us (the
// first passes are the long ones); 16385 packed tokens, 16/4 heads of 128, buckets: dq 266 us, dk and dv 244 us at best (530 us
// with four waves a workgroup and tiles in the order of the documents), table 9 us, plan 7 us.  dk and dv of small fp32 problems at 128 wide spill 33 to 92
// registers, and are faster than the kernel that does not (1024 tokens, 16 heads: 139 us with the join against 266).
#include <type_traits>

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

// A thread's share (every `step`-th distance from `from` on) of a bucket's cells in the sums by relative position;
// interior only: distances of max_distance and more are summed apart.
__device__ __forceinline__ float fold_bucket(const AttnBuckets& b, const float* sums, int bucket, int from, int step) {
    const int n = b.nborders + 1, in = bucket % n;
    const bool behind = b.both && bucket >= n;
    const int lo = in == 0 ? 0 : b.borders[in - 1], hi = in == n - 1 ? b.max_distance : b.borders[in];
    float v = 0.f;
    for (int d = lo + from; d < hi; d += step)
        if (!behind || d > 0) v += sums[b.max_distance + (behind ? d : -d)];
    if (!b.both && in == 0)
        for (int d = 1 + from; d < b.max_distance; d += step) v += sums[b.max_distance + d];
    return v;
}

// How a workgroup shares its work.  (Paired key gradients at 64-wide heads, whose sums leave room for two waves a SIMD
// anyway: 452 us against 350.)
enum Share {
    kAlone = 0,   // four waves, 32 rows (keys) each
    kSplit = 1,   // four waves on the same 32 (see kOwn)
    kPaired = 2,  // eight waves, two on the same 32, each with half of a streamed tile, and the operands of the workgroup's
                  // own rows in LDS: the sums of 128-wide heads alone fill half a SIMD's registers, and so two waves
                  // still fit on each
};

// Adds the sums of a pair's second wave to its first's, through a buffer of the pair's own.
template <int DT> __device__ __forceinline__ void add_second(f32x16 (&acc)[DT], float* over, int second, int lane) {
    f32x4* at = reinterpret_cast<f32x4*>(over) + lane;
    if (second) {
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int r = 0; r < 16; r += 4)
                at[(4 * d + r / 4) * kWave] = f32x4{acc[d][r], acc[d][r + 1], acc[d][r + 2], acc[d][r + 3]};
    }
    __syncthreads();
    if (!second) {
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const f32x4 x = at[(4 * d + r / 4) * kWave];
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[d][r + e] += x[e];
            }
    }
    __syncthreads();
}

// How dq gets rid of what a bf16 y leaves in D: with the sum of p k beside the sum of dS k (MEAN), or with a pass of its own
// for D before (PASS).  dq with the sum, with the pass and with neither, us, bf16, 16385 tokens in 32 documents, 16/4 heads
// (4 x 2048 tokens, 8 heads):
//     64 wide  80 (n/a), 106, 63                          with buckets and their gradient  184 (144), 165 (211), 126 (128)
//     128 wide 230 (131), 209 (231), 139 (135)            with buckets and their gradient  359, 269, 221
template <typename T, int D, int BIAS> constexpr bool kTakesPass = sizeof(T) == 2 && D == 128 && BIAS == kBiasBuckets;
template <typename T, int D, int BIAS> constexpr bool kTakesMean = sizeof(T) == 2 && !kTakesPass<T, D, BIAS>;

// Waves a SIMD that the sums and operands in registers leave room for.
template <int ROW, int D, bool MEAN, int SHARE>
constexpr int kQueryWaves = SHARE != kAlone || ROW >= 512 ? 1 : ROW == 256 || (MEAN && D == 64) ? 2 : 3;

template <typename T, int D, bool CAP, int BIAS, int SHARE>
__global__ void __launch_bounds__(SHARE == kPaired ? 2 * kThreads : kThreads,
                                  (kQueryWaves<(int)sizeof(T) * D, D, kTakesMean<T, D, BIAS>, SHARE>))
    attn_dq_kernel(AttnParams p) {
    using O = Op<T>;
    using L = Tile<T, D>;
    using Frag = typename O::Frag;
    constexpr bool SPLIT = SHARE == kSplit, PAIRED = SHARE == kPaired, MEAN = kTakesMean<T, D, BIAS>;
    static_assert(!PAIRED || BIAS != kBiasBuckets, "the sums by distance are those of four waves");
    constexpr int OWN = kOwn<SPLIT>, KT = SPLIT ? 32 : O::kKT, NT = D / O::kK, DT = D / 32, PK = 32 / O::kK;
    constexpr int NS = PAIRED ? 1 : KT / 32;  // 32-key blocks of a tile that are this wave's
    constexpr int BLOCK = PAIRED ? 2 * kThreads : kThreads;
    constexpr int ELEMS = (SPLIT ? kWaves : 1) * KT * D;
    constexpr bool DOUBLE = !SPLIT || ELEMS * sizeof(T) <= 32768;
    __shared__ __attribute__((aligned(16))) T k_a[ELEMS];
    __shared__ __attribute__((aligned(16))) T v_a[ELEMS];
    __shared__ __attribute__((aligned(16))) T k_b[DOUBLE ? ELEMS : 8];
    __shared__ __attribute__((aligned(16))) T v_b[DOUBLE ? ELEMS : 8];
    __shared__ __attribute__((aligned(16))) T q_own[PAIRED ? OWN * D : 8];
    __shared__ __attribute__((aligned(16))) T g_own[PAIRED ? OWN * D : 8];
    __shared__ float off_by[SPLIT || PAIRED ? BLOCK / 2 : 1];
    extern __shared__ float extra[];

    int slot, unit;
    work_item(blockIdx.x, p.q_slots, (uint32_t)p.H / (uint32_t)p.pack, slot, unit);
    const Span sp = find_span(p, slot, OWN, false);
    const int head0 = unit * p.pack;
    const bool grad = BIAS == kBiasBuckets && p.dtable != nullptr;
    float* part = grad ? p.table_part + ((int64_t)sp.slot * p.H + head0) * p.bk.total : nullptr;
    if (sp.tile < 0) {
        if (grad)
            for (int i = threadIdx.x; i < p.bk.total; i += kThreads) part[i] = 0.f;
        return;
    }
    const int kvh = (int)((uint32_t)head0 / ((uint32_t)p.H / (uint32_t)p.Hk));
    const int lane = threadIdx.x % kWave, half = lane / 32;
    const int all_waves = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int wave = all_waves % kWaves, n_own = all_waves / kWaves;  // (PAIRED: which 32 keys of a tile)
    const int shift = sp.lk - sp.lq;
    int prefix = 0;
    if (p.prefix) prefix = (int)clamp64(p.prefix[sp.seq], 0, sp.lk);
    auto limit = [&](int i) { return p.causal ? max(min(max(i + shift + 1, prefix), sp.lk), 0) : sp.lk; };
    const int row0 = sp.tile * OWN + (SPLIT ? 0 : wave * 32), row = row0 + lane % 32;
    auto query_of = [&](int r) { return (int)((uint32_t)r / (uint32_t)p.pack); };
    const int query = query_of(min(row, sp.rows - 1)), head = head0 + min(row, sp.rows - 1) - query * p.pack;
    const int wg_limit = limit(query_of(min(sp.tile * OWN + OWN, sp.rows) - 1));
    const int ntiles = (wg_limit + KT - 1) / KT;
    const int my_limit = row < sp.rows ? limit(query) : 0;
    const int wave_most = row0 < sp.rows ? limit(query_of(min(row0 + 32, sp.rows) - 1)) : 0;
    const int wave_least = limit(query_of(row0));

    const T* kg = static_cast<const T*>(p.k) + sp.k0 * p.k_stride + (int64_t)kvh * D;
    const T* vg = static_cast<const T*>(p.v) + sp.k0 * p.v_stride + (int64_t)kvh * D;
    Feed<T, D, KT, SPLIT ? kWave : BLOCK> kf, vf;
    kf.init(p.k_stride);
    vf.init(p.v_stride);
    const int at = SPLIT ? wave * KT * D : 0;
    T *ka = k_a + at, *va = v_a + at, *kb = k_b + (DOUBLE ? at : 0), *vb = v_b + (DOUBLE ? at : 0);
    auto fetch = [&](T* ks, T* vs, int t) __attribute__((always_inline)) {
        kf.load(ks, kg, t * KT, sp.lk - t * KT);
        vf.load(vs, vg, t * KT, sp.lk - t * KT);
    };
    const int t0 = SPLIT ? wave : 0, dt = SPLIT ? kWaves : 1;
    if (t0 < ntiles) fetch(ka, va, t0);

    const int64_t mine = (sp.q0 + query) * p.H + head;  // this lane's (query, head)
    Frag qf[PAIRED ? 1 : NT], gf[PAIRED ? 1 : NT];
    float delta = 0.f;
    {
        const T* qg = static_cast<const T*>(p.q) + (sp.q0 + query) * p.q_stride + (int64_t)head * D;
        const T* gg = static_cast<const T*>(p.dy) + mine * D;
        const T* yg = static_cast<const T*>(p.y) + mine * D;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int e0 = (2 * t + half) * O::kE;
            const Frag g = __builtin_bit_cast(Frag, ld16(gg + e0)), yf = __builtin_bit_cast(Frag, ld16(yg + e0));
            if constexpr (PAIRED) {  // (a pair's first wave keeps the queries, its second dy)
                const int own = L::at(32 * wave + lane % 32, 2 * t + half);
                if (n_own == 0) st16(q_own + own, ld16(qg + e0));
                else st16(g_own + own, __builtin_bit_cast(uint4, g));
            } else {
                qf[t] = __builtin_bit_cast(Frag, ld16(qg + e0));
                gf[t] = g;
            }
#pragma unroll
            for (int e = 0; e < O::kE; ++e) delta += (float)g[e] * (float)yf[e];
        }
    }
    delta += other_half(delta);
    float lse2 = p.lse[mine] * kLog2e;
    // a row that sees nothing, and the tile's rows past the last query: all their weights are zero
    if (lse2 == -INFINITY || row >= sp.rows) lse2 = INFINITY;

    Score sc;
    sc.init<T>(p.scale, p.cap, CAP, BIAS == kBiasNone);
    float slope2 = 0.f;
    if constexpr (BIAS == kBiasSlopes) slope2 = p.slopes[head] * kLog2e;
    const int md = p.bk.max_distance, reach = 2 * md + 1;
    float* lut = extra;
    float* sums = extra + reach + wave * reach;                                 // by relative position
    float* block = extra + (1 + kWaves) * reach + wave * kDiagBlock;            // dS [key][query]
    float* far = extra + (1 + kWaves) * reach + kWaves * kDiagBlock;            // [2][kWaves]
    if constexpr (BIAS == kBiasBuckets) {
        fill_bias(lut, p, head0);
        if (grad)
            for (int i = lane; i < reach; i += kWave) sums[i] = 0.f;
    }
    // the row's sum of dS (before the cap's derivative), and that of far cells below and above the reach
    float row_ds = 0.f, far_lo = 0.f, far_hi = 0.f, far_lo_p = 0.f, far_hi_p = 0.f;  // (and of their p)
    const int qpos = query + shift;

    f32x16 acc[DT], mean[MEAN ? DT : 1];  // sums of dS k and of p k
#pragma unroll
    for (int d = 0; d < DT; ++d) acc[d] = f32x16{};
#pragma unroll
    for (int d = 0; d < (MEAN ? DT : 1); ++d) mean[d] = f32x16{};

    auto settle = [&]() __attribute__((always_inline)) {
        __builtin_amdgcn_s_waitcnt(SPLIT ? kAllDone : kLoadsDone);
        if constexpr (SPLIT) __builtin_amdgcn_wave_barrier(); else lds_barrier();
    };
    // p and dS of 32 keys from kn on, before the cap's derivative, which is returned in `slope`, or with no bias and
    // `whole` already in both (dS before it is then in row_ds); true: some are nearer than the table's reach
    typename L::Lanes z(lane);
    auto q_frag = [&](int i) { return PAIRED ? L::rows(q_own, 32 * wave, i, z) : qf[PAIRED ? 0 : i]; };
    auto g_frag = [&](int i) { return PAIRED ? L::rows(g_own, 32 * wave, i, z) : gf[PAIRED ? 0 : i]; };
    auto weights = [&](const T* kt, const T* vt, int n, int kn, f32x16& s, f32x16& ds, f32x16& slope, bool whole) __attribute__((always_inline)) {
        z.renew();
        f32x16 x[1] = {f32x16{}}, dp;
#pragma unroll
        for (int r = 0; r < 16; ++r) dp[r] = -delta;  // the accumulator starts at -D: dP - D at no cost
#pragma unroll
        for (int i = 0; i < NT; ++i) x[0] = O::mma(L::rows(kt, 32 * n, i, z), q_frag(i), x[0]);
#pragma unroll
        for (int i = 0; i < NT; ++i) dp = O::mma(L::rows(vt, 32 * n, i, z), g_frag(i), dp);
        // (left to itself the schedule holds more than there are registers for)
        if constexpr (PAIRED) __builtin_amdgcn_sched_barrier(0);
        if constexpr (CAP) {
            sc.template capped<T>(x);
            if constexpr (BIAS != kBiasNone) {
#pragma unroll
                for (int r = 0; r < 16; ++r) slope[r] = sc.slope(x[0][r]);
            }
        }
        const bool near = add_bias<BIAS, 1>(x, CAP ? 1.f : sc.a, slope2, lut, md, kn + 4 * half - qpos, kn - (row0 + 31 + shift),
                                            kn + 31 - (row0 + shift));
        if (kn + 32 > wave_least) {
            const int left = my_limit - kn - 4 * half;
#pragma unroll
            for (int r = 0; r < 16; ++r) x[0][r] = acc_row(r) < left ? x[0][r] : sc.none;
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            s[r] = exp2_hw(!CAP && BIAS == kBiasNone ? __builtin_fmaf(x[0][r], sc.a, -lse2) : x[0][r] - lse2);
            // (without a bias the capped score is still there to take the derivative from)
            if constexpr (CAP && BIAS == kBiasNone) {
                if (whole) {
                    if constexpr (MEAN) row_ds = __builtin_fmaf(s[r], dp[r], row_ds);
                    s[r] *= sc.slope(x[0][r]);
                }
            }
            ds[r] = s[r] * dp[r];
        }
        return near;
    };
    // Sums of dS along the diagonals of 16 keys x 32 queries at a time: lane j takes relative position base + j, from the
    // corner key 0, query 31 on.
    auto by_distance = [&](const f32x16& ds, int kn) __attribute__((always_inline)) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int r = 0; r < 8; ++r) block[(acc_row(r) + 4 * half) * kDiagStride + lane % 32] = ds[8 * b + r];
            __builtin_amdgcn_wave_barrier();
            const int off = lane - 31, rel = kn + 16 * b - (row0 + shift) + off;
            float add = 0.f;
#pragma unroll
            for (int key = 0; key < kDiagRows; ++key) {
                const int q = key - off;
                const float x = block[key * kDiagStride + min(max(q, 0), 31)];
                add += q >= 0 && q < 32 ? x : 0.f;
            }
            if (lane < 31 + kDiagRows) {
                if (rel <= -md) far_lo += add;
                else if (rel >= md) far_hi += add;
                else sums[rel + md] += add;
            }
            __builtin_amdgcn_wave_barrier();
        }
    };
    // (ONLY_D: the first of two passes, for the sum of dS alone)
    auto step = [&](auto only_d, const T* kt, const T* vt, T* kn_, T* vn_, int t) __attribute__((always_inline)) {
        constexpr bool ONLY_D = decltype(only_d)::value;
        const int k0 = t * KT;
        if (DOUBLE && t + dt < ntiles) fetch(kn_, vn_, t + dt);
        if (k0 < wave_most) {
            // (one half of a tile after the other: both at once take the registers of one more wave a SIMD)
#pragma unroll 1
            for (int j = 0; j < NS; ++j) {
                const int n = PAIRED ? n_own : j, kn = k0 + 32 * n;
                f32x16 s, ds, slope;
                const bool near = weights(kt, vt, n, kn, s, ds, slope, !ONLY_D);
                if constexpr (ONLY_D || (MEAN && CAP && BIAS == kBiasSlopes)) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) row_ds += ds[r];
                }
                if constexpr (ONLY_D) continue;
                if constexpr (BIAS == kBiasBuckets && !MEAN) {
                    if (grad) {
                        if (near) {
                            by_distance(ds, kn);
                        } else {
                            float a = 0.f;
#pragma unroll
                            for (int r = 0; r < 16; ++r) a += ds[r];
                            const bool above = kn >= row0 + shift;
                            far_lo += above ? 0.f : a;
                            far_hi += above ? a : 0.f;
                        }
                    }
                }
                if constexpr (BIAS == kBiasBuckets && MEAN) {
                    if (grad || CAP) {
                        float a = 0.f, b = 0.f;
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            a += ds[r];
                            b += s[r];
                        }
                        row_ds += a;
                        const bool above = kn >= row0 + shift;
                        far_lo += near || above ? 0.f : a;
                        far_lo_p += near || above ? 0.f : b;
                        far_hi += near || !above ? 0.f : a;
                        far_hi_p += near || !above ? 0.f : b;
                    }
                }
                if constexpr (CAP && BIAS != kBiasNone) {
                    ds *= slope;
                    if constexpr (MEAN) s *= slope;
                }
#pragma unroll
                for (int kk = 0; kk < PK; ++kk) {
                    const Frag sf = O::pack(ds, kk), pf = O::pack(s, kk);
                    if constexpr (MEAN && !CAP) {
                        if (!grad) row_ds = sum_of(sf, row_ds);
                    }
#pragma unroll
                    for (int d = 0; d < DT; ++d) {
                        const Frag kf = L::cols(kt, 32 * n, kk, 32 * d, z);
                        acc[d] = O::mma(kf, sf, acc[d]);
                        if constexpr (MEAN) mean[d] = O::mma(kf, pf, mean[d]);
                    }
                }
            }
        }
        settle();
        if (!DOUBLE && t + dt < ntiles) {
            fetch(kn_, vn_, t + dt);
            settle();
        }
    };
    auto pass = [&](auto only_d) __attribute__((always_inline)) {
        settle();
        for (int t = t0; t < ntiles; t += 2 * dt) {
            step(only_d, ka, va, DOUBLE ? kb : ka, DOUBLE ? vb : va, t);
            if (t + dt < ntiles) step(only_d, DOUBLE ? kb : ka, DOUBLE ? vb : va, ka, va, t + dt);
        }
    };
    // the sum of a row's dS over all its keys, which its D is off by
    auto row_sum = [&]() __attribute__((always_inline)) {
        row_ds += other_half(row_ds);
        if constexpr (SPLIT || PAIRED) {
            if (half == 0) off_by[32 * all_waves + lane] = row_ds;
            __syncthreads();
            row_ds = 0.f;
#pragma unroll
            for (int w = 0; w < BLOCK / kWave; ++w) row_ds += SPLIT || w % kWaves == wave ? off_by[32 * w + lane % 32] : 0.f;
        }
        delta += row_ds;
    };
    if constexpr (SPLIT && BIAS == kBiasBuckets) __syncthreads();
    if constexpr (kTakesPass<T, D, BIAS>) {
        pass(std::true_type{});
        row_sum();
        if (t0 < ntiles) fetch(ka, va, t0);
    }
    pass(std::false_type{});
    if constexpr (MEAN) {
        row_sum();
#pragma unroll
        for (int d = 0; d < DT; ++d) acc[d] -= row_ds * mean[d];
    }

    if constexpr (SPLIT) {
        __syncthreads();
        Join<T, D>::keep(k_a, v_a, acc, lane, wave);
        __syncthreads();
        for (int i = threadIdx.x; i < 32 * (D / 4); i += kThreads) {
            const int r = i / (D / 4), d4 = i % (D / 4);
            if (row0 + r >= sp.rows) break;
            const f32x4 v = Join<T, D>::sum(k_a, v_a, r, d4, nullptr) * p.scale;
            const int q = query_of(row0 + r);
            store4(static_cast<T*>(p.dq) + ((sp.q0 + q) * p.H + head0 + row0 + r - q * p.pack) * D + 4 * d4, v[0], v[1], v[2], v[3]);
        }
    } else {
        if constexpr (PAIRED) {
            static_assert(!PAIRED || ELEMS * sizeof(T) == 32 * D * 4, "a tile's buffer holds one wave's sums");
            add_second(acc, reinterpret_cast<float*>(wave == 0 ? k_a : wave == 1 ? v_a : wave == 2 ? k_b : v_b), n_own, lane);
        }
        if (row < sp.rows && n_own == 0) {
            T* out = static_cast<T*>(p.dq) + mine * D;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int r = 0; r < 16; r += 8) store_rows(out + 32 * d, acc[d], r, half, p.scale);
        }
    }
    if (row < sp.rows && half == 0 && (SPLIT ? wave : n_own) == 0) p.delta[mine] = delta;
    if constexpr (BIAS == kBiasBuckets) {
        if (!grad) return;
        if constexpr (MEAN) {
            // D is exact now: far cells are put right by the sums of their p, and the tiles with a relative position inside
            // the reach of any of the workgroup's queries are visited again
            far_lo -= row_ds * far_lo_p;
            far_hi -= row_ds * far_hi_p;
            const int q_first = sp.tile * OWN + shift, q_last = q_first + OWN - 1;
            const int n0 = max(q_first - md, 0) / KT, n1 = min(ntiles, q_last + md < 0 ? 0 : (q_last + md) / KT + 1);
            if constexpr (SPLIT) __syncthreads();  // (the tiles are free again)
            for (int t = n0 + t0; t < n1; t += dt) {
                const int k0 = t * KT;
                fetch(ka, va, t);
                settle();
                if (k0 < wave_most) {
#pragma unroll 1
                    for (int n = 0; n < NS; ++n) {
                        const int kn = k0 + 32 * n;
                        if (kn + 31 - (row0 + shift) <= -md || kn - (row0 + 31 + shift) >= md) continue;
                        f32x16 s, ds, slope;
                        weights(ka, va, n, kn, s, ds, slope, false);
                        by_distance(ds, kn);
                    }
                }
                settle();
            }
        }
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
        float* all = extra + reach;
        for (int i = threadIdx.x; i < reach; i += kThreads) {
            float v = all[i];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) v += all[w * reach + i];
            all[i] = v;
        }
        __syncthreads();
        // as many lanes to a bucket as there are, in powers of two
        const int lanes = 1 << (31 - __clz(kThreads / p.bk.total)), i = (int)threadIdx.x / lanes;
        const int per = min(lanes, kWave);
        if (i < p.bk.total) {
            float v = fold_bucket(p.bk, all, i, threadIdx.x % lanes, lanes);
            for (int off = per / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
            if (lanes <= kWave) {
                if (threadIdx.x % lanes == 0) {
                    for (int w = 0; w < kWaves; ++w) {
                        if (i == p.bk.nborders) v += far[w];  // the last bucket of the first direction
                        if (i == (p.bk.both ? p.bk.total - 1 : 0)) v += far[kWaves + w];
                    }
                    part[i] = v;
                }
            } else if (lane == 0) {  // (two buckets: two waves each)
                block[0] = v;
            }
        }
        if (lanes > kWave) {
            __syncthreads();
            if ((int)threadIdx.x < p.bk.total) {
                const int b = threadIdx.x, waves = lanes / kWave;
                float v = 0.f;
                for (int w = 0; w < waves; ++w) v += extra[(1 + kWaves) * reach + (b * waves + w) * kDiagBlock];
                for (int w = 0; w < kWaves; ++w) {
                    if (b == p.bk.nborders) v += far[w];
                    if (b == (p.bk.both ? p.bk.total - 1 : 0)) v += far[kWaves + w];
                }
                part[b] = v;
            }
        }
    }
}

// The slots of the query (block 0) and key axis (block 1) in order of their work, most first: a counting sort by
// the number of 64-row steps, empty slots last.  The order among equals varies from run to run, and is of no
// consequence: a workgroup's results are its own, and lie where its tile does.
constexpr int kPlanThreads = 1024, kPlanBins = 2048;
__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(AttnParams p, int q_own, int k_own) {
    __shared__ int bins[kPlanBins];
    __shared__ int scan[kPlanThreads];
    const bool keys = blockIdx.x == 1;
    const int own = keys ? k_own : q_own;
    if (own == 0) return;
    const int64_t* cu = keys ? p.cu_k : p.cu_q;
    int2* plan = keys ? p.plan_k : p.plan_q;
    const int tq = (int)p.total_q, tk = (int)p.total_k, total = keys ? tk : tq, nseq = (int)p.nseq;
    const int pack = keys ? 1 : p.pack;
    const int slots = (int)((int64_t)total * pack / own) + nseq;
    auto start = [&](int s) { return (int)((int64_t)offset_at(cu, s, total) * pack / own) + s; };
    int2* raw = plan + slots;  // (sequence, tile) by slot
    for (int i = threadIdx.x; i < kPlanBins; i += kPlanThreads) bins[i] = 0;
    __syncthreads();
    auto bin_of = [&](int s, int tile) {
        const int q0 = offset_at(p.cu_q, s, tq), lq = max(offset_at(p.cu_q, s + 1, tq) - q0, 0);
        const int k0 = offset_at(p.cu_k, s, tk), lk = max(offset_at(p.cu_k, s + 1, tk) - k0, 0), shift = lk - lq;
        const int prefix = p.prefix ? (int)clamp64(p.prefix[s], 0, lk) : 0;
        int rows;
        if (keys) rows = lq - (!p.causal || tile * own < prefix ? 0 : max(tile * own - shift, 0));
        else rows = p.causal ? max(min(max(min((tile * own + own - 1) / pack + 1, lq) + shift, prefix), lk), 0) : lk;
        return kPlanBins - 1 - min(max((rows + 63) / 64, 0) + 1, kPlanBins - 1);
    };
    for (int slot = threadIdx.x; slot < slots; slot += kPlanThreads) {
        int lo = 0, n = nseq;  // the last sequence that starts at this slot or before
        while (n > 1) {
            const int mid = n / 2;
            if (start(lo + mid) <= slot) {
                lo += mid;
                n -= mid;
            } else {
                n = mid;
            }
        }
        int tile = slot - start(lo);
        const int64_t len = (int64_t)(offset_at(cu, lo + 1, total) - offset_at(cu, lo, total)) * pack;
        if (tile < 0 || (int64_t)tile * own >= len) tile = -1;
        raw[slot] = int2{tile < 0 ? slot : lo, tile};
        atomicAdd(&bins[tile < 0 ? kPlanBins - 1 : bin_of(lo, tile)], 1);
    }
    __syncthreads();
    // exclusive sums of the bins, two a thread
    const int a = bins[2 * threadIdx.x], b = bins[2 * threadIdx.x + 1];
    scan[threadIdx.x] = a + b;
    __syncthreads();
    for (int off = 1; off < kPlanThreads; off <<= 1) {
        const int v = threadIdx.x >= off ? scan[threadIdx.x - off] : 0;
        __syncthreads();
        scan[threadIdx.x] += v;
        __syncthreads();
    }
    const int before = scan[threadIdx.x] - a - b;
    bins[2 * threadIdx.x] = before;
    bins[2 * threadIdx.x + 1] = before + a;
    __syncthreads();
    for (int slot = threadIdx.x; slot < slots; slot += kPlanThreads) {
        const int2 e = raw[slot];
        const int at = atomicAdd(&bins[e.y < 0 ? kPlanBins - 1 : bin_of(e.x, e.y)], 1);
        plan[slots - 1 - at] = e;  // (workgroups take slots from the last one down)
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

template <typename T, int D, bool CAP, int BIAS, int SHARE>
__global__ void __launch_bounds__(SHARE == kPaired ? 2 * kThreads : kThreads, SHARE != kAlone || sizeof(T) * D >= 256 ? 1 : 2)
    attn_dkv_kernel(AttnParams p) {
    using O = Op<T>;
    using L = Tile<T, D>;
    using Frag = typename O::Frag;
    constexpr bool SPLIT = SHARE == kSplit, PAIRED = SHARE == kPaired;
    constexpr int OWN = kOwn<SPLIT>, QT = SPLIT ? 32 : O::kKT, NT = D / O::kK, DT = D / 32, PK = 32 / O::kK;
    constexpr int NS = PAIRED ? 1 : QT / 32;  // 32-query blocks of a tile that are this wave's
    constexpr int BLOCK = PAIRED ? 2 * kThreads : kThreads;
    constexpr int COPIES = SPLIT ? kWaves : 1, ELEMS = COPIES * QT * D, THREADS = SPLIT ? kWave : BLOCK;
    constexpr bool DOUBLE = !SPLIT || ELEMS * sizeof(T) <= 32768;
    __shared__ __attribute__((aligned(16))) T q_a[ELEMS];
    __shared__ __attribute__((aligned(16))) T g_a[ELEMS];
    __shared__ __attribute__((aligned(16))) T q_b[DOUBLE ? ELEMS : 8];
    __shared__ __attribute__((aligned(16))) T g_b[DOUBLE ? ELEMS : 8];
    __shared__ __attribute__((aligned(16))) T k_own[PAIRED ? OWN * D : 8];
    __shared__ __attribute__((aligned(16))) T v_own[PAIRED ? OWN * D : 8];
    __shared__ __attribute__((aligned(16))) float stat[2][COPIES][2][QT];  // [buffer][wave][lse in log2 units, D][query]
    extern __shared__ float extra[];
    float* lut = extra;

    int slot, kvh;
    work_item(blockIdx.x, p.k_slots, SPLIT ? p.Hk * p.parts : p.Hk, slot, kvh);
    const int part = SPLIT ? kvh % p.parts : 0;
    if constexpr (SPLIT) kvh /= p.parts;
    if (!p.plan_k) slot = p.k_slots - 1 - slot;  // under a causal mask the first keys are seen by the most queries
    const Span sp = find_span(p, slot, OWN, true);
    if (sp.tile < 0) return;
    const int group = p.H / p.Hk;
    const int lane = threadIdx.x % kWave, half = lane / 32;
    const int all_waves = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int wave = all_waves % kWaves, n_own = all_waves / kWaves;  // (PAIRED: which 32 queries of a tile)
    const int shift = sp.lk - sp.lq;
    int prefix = 0;
    if (p.prefix) prefix = (int)clamp64(p.prefix[sp.seq], 0, sp.lk);

    // queries [first(j), lq) see key j
    auto first = [&](int j) { return !p.causal || j < prefix ? 0 : max(j - shift, 0); };
    const int row0 = sp.tile * OWN + (SPLIT ? 0 : wave * 32), key = row0 + lane % 32;
    const int t0 = first(sp.tile * OWN) / QT, t1 = (sp.lq + QT - 1) / QT;
    const int my_first = key < sp.lk ? first(key) : sp.lq;
    const int wave_least = row0 < sp.lk ? first(row0) : sp.lq;  // the earliest query that any key of the wave meets
    const int wave_most = row0 + 32 <= sp.lk ? first(row0 + 31) : sp.lq;  // from here on every key meets every query
    const int per_head = max(t1 - t0, 0), all_tiles = per_head * group;
    // (SPLIT: this workgroup's part of them)
    const int first_tile = SPLIT ? (int)((int64_t)all_tiles * part / p.parts) : 0;
    const int ntiles = SPLIT ? (int)((int64_t)all_tiles * (part + 1) / p.parts) : all_tiles;

    Feed<T, D, QT, THREADS> qf, gf;
    qf.init(p.q_stride);
    gf.init((int64_t)p.H * D);
    const int tid = SPLIT ? lane : (int)threadIdx.x;
    // a tile's queries and dy go straight to LDS; its statistics (threads 0 .. QT - 1: lse, the next QT: D) wait in a
    // register until then.  They are what the accumulators of S and dP start from: -D, and where the scores
    // stay raw products until the exponential, -lse in their units.
    constexpr bool RAW = !CAP && BIAS == kBiasNone;
    Score sc;
    sc.init<T>(p.scale, p.cap, CAP, BIAS == kBiasNone);
    const float unit = RAW ? -kLog2e / sc.a : kLog2e;
    float sb = 0.f;
    auto fetch = [&](T* qs, T* gs, int it) {
        const int head = kvh * group + it / per_head, row = (t0 + it % per_head) * QT;
        qf.load(qs, static_cast<const T*>(p.q) + sp.q0 * p.q_stride + (int64_t)head * D, row, sp.lq - row);
        gf.load(gs, static_cast<const T*>(p.dy) + (sp.q0 * p.H + head) * D, row, sp.lq - row);
        if (tid < 2 * QT) {
            const int64_t at = (sp.q0 + min(row + tid % QT, sp.lq - 1)) * p.H + head;
            sb = tid < QT ? p.lse[at] : -p.delta[at];
            // (a query that sees nothing: all its weights are zero)
            if (tid < QT) sb = (sb == -INFINITY ? INFINITY : sb) * unit;
        }
    };
    const int copy = SPLIT ? wave : 0;
    auto settle = [&](int buf) {  // (every thread's statistics of the next tile, where it has fetched any)
        if (tid < 2 * QT) stat[buf][copy][tid / QT][tid % QT] = sb;
        __builtin_amdgcn_s_waitcnt(SPLIT ? kAllDone : kLoadsDone);
        if constexpr (SPLIT) __builtin_amdgcn_wave_barrier(); else lds_barrier();
    };
    const int at = copy * QT * D;
    T *qa = q_a + at, *ga = g_a + at, *qb = q_b + (DOUBLE ? at : 0), *gb = g_b + (DOUBLE ? at : 0);
    // SPLIT: a wave takes every fourth tile
    const int i0 = SPLIT ? first_tile + wave : 0, di = SPLIT ? kWaves : 1;
    if (i0 < ntiles) fetch(qa, ga, i0);

    Frag kf[PAIRED ? 1 : NT], vf[PAIRED ? 1 : NT];
    if constexpr (PAIRED) {
        Feed<T, D, OWN, BLOCK> own;
        const int row = sp.tile * OWN;
        own.init(p.k_stride);
        own.load(k_own, static_cast<const T*>(p.k) + sp.k0 * p.k_stride + (int64_t)kvh * D, row, sp.lk - row);
        own.init(p.v_stride);
        own.load(v_own, static_cast<const T*>(p.v) + sp.k0 * p.v_stride + (int64_t)kvh * D, row, sp.lk - row);
    } else {
        const int64_t krow = sp.k0 + min(key, sp.lk - 1);
        const T* kg = static_cast<const T*>(p.k) + krow * p.k_stride + (int64_t)kvh * D;
        const T* vg = static_cast<const T*>(p.v) + krow * p.v_stride + (int64_t)kvh * D;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            kf[t] = __builtin_bit_cast(Frag, ld16(kg + (2 * t + half) * O::kE));
            vf[t] = __builtin_bit_cast(Frag, ld16(vg + (2 * t + half) * O::kE));
        }
    }
    typename L::Lanes z(lane);
    auto k_frag = [&](int i) { return PAIRED ? L::rows(k_own, 32 * wave, i, z) : kf[PAIRED ? 0 : i]; };
    auto v_frag = [&](int i) { return PAIRED ? L::rows(v_own, 32 * wave, i, z) : vf[PAIRED ? 0 : i]; };
    const int md = p.bk.max_distance;
    if constexpr (BIAS == kBiasBuckets) {
        // one head's bias, refilled where the head changes; SPLIT: the waves are on different heads at a time,
        // so that every head's is there at once
        if constexpr (SPLIT)
            for (int h = 0; h < group; ++h) fill_bias(lut + h * (2 * md + 1), p, kvh * group + h);
        else fill_bias(lut, p, kvh * group);
    }

    f32x16 dk[DT], dv[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) dk[d] = dv[d] = f32x16{};

    auto step = [&](const T* qt, const T* gt, T* qn_, T* gn_, int it, int buf) {
        const int h = it / per_head, head = kvh * group + h, q0 = (t0 + it % per_head) * QT;
        const float* bias = lut;
        if constexpr (BIAS == kBiasBuckets) {
            if constexpr (SPLIT) {
                bias = lut + h * (2 * md + 1);
            } else if (h > 0 && it % per_head == 0) {  // (the barrier before this: nobody reads the old one)
                fill_bias(lut, p, head);
                __syncthreads();
            }
        }
        float slope2 = 0.f;
        if constexpr (BIAS == kBiasSlopes) slope2 = p.slopes[head] * kLog2e;
        if (DOUBLE && it + di < ntiles) fetch(qn_, gn_, it + di);
        if (q0 + QT > wave_least) {
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                const int n = PAIRED ? n_own : j;
                if constexpr (PAIRED) z.renew();
                const float* ls = &stat[buf][copy][0][32 * n + 4 * half];
                const float* de = &stat[buf][copy][1][32 * n + 4 * half];
                f32x16 s[1] = {f32x16{}}, dp;
#pragma unroll
                for (int r = 0; r < 16; r += 4) {
                    const f32x4 dl = as_f32x4(ld16(de + acc_row(r)));
#pragma unroll
                    for (int e = 0; e < 4; ++e) dp[r + e] = dl[e];
                    if constexpr (RAW) {
                        const f32x4 lv = as_f32x4(ld16(ls + acc_row(r)));
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[0][r + e] = lv[e];
                    }
                }
#pragma unroll
                for (int i = 0; i < NT; ++i) s[0] = O::mma(L::rows(qt, 32 * n, i, z), k_frag(i), s[0]);
#pragma unroll
                for (int i = 0; i < NT; ++i) dp = O::mma(L::rows(gt, 32 * n, i, z), v_frag(i), dp);
                const int qn = q0 + 32 * n;
                f32x16 slope;
                if constexpr (CAP) {
                    sc.template capped<T>(s);
                    if constexpr (BIAS != kBiasNone) {
#pragma unroll
                        for (int r = 0; r < 16; ++r) slope[r] = sc.slope(s[0][r]);
                    }
                }
                // (of register 0; later queries are further back)
                add_bias<BIAS, -1>(s, CAP ? 1.f : sc.a, slope2, bias, md, key - (qn + shift + 4 * half), row0 - (qn + 31 + shift),
                                   row0 + 31 - (qn + shift));
                if (qn < wave_most || qn + 32 > sp.lq) {
                    const int lo = my_first - qn - 4 * half, hi = sp.lq - qn - 4 * half;
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[0][r] = acc_row(r) >= lo && acc_row(r) < hi ? s[0][r] : sc.none;
                }
#pragma unroll
                for (int r = 0; r < 16; r += 4) {
                    f32x4 lv{};
                    if constexpr (!RAW) lv = as_f32x4(ld16(ls + acc_row(r)));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x = s[0][r + e];
                        s[0][r + e] = exp2_hw(RAW ? x * sc.a : x - lv[e]);
                        dp[r + e] *= s[0][r + e];
                        if constexpr (CAP && BIAS == kBiasNone) dp[r + e] *= sc.slope(x);
                    }
                }
                if constexpr (CAP && BIAS != kBiasNone) dp *= slope;
#pragma unroll
                for (int kk = 0; kk < PK; ++kk) {
                    const Frag pf = O::pack(s[0], kk), sf = O::pack(dp, kk);
#pragma unroll
                    for (int d = 0; d < DT; ++d) {
                        dv[d] = O::mma(L::cols(gt, 32 * n, kk, 32 * d, z), pf, dv[d]);
                        dk[d] = O::mma(L::cols(qt, 32 * n, kk, 32 * d, z), sf, dk[d]);
                    }
                }
            }
        }
        if constexpr (!DOUBLE) {
            settle(1);  // (a buffer that nobody reads)
            if (it + di < ntiles) fetch(qn_, gn_, it + di);
            settle(0);
        } else {
            settle(buf ^ 1);
        }
    };
    settle(0);
    if constexpr (SPLIT && BIAS == kBiasBuckets) __syncthreads();
    for (int it = i0; it < ntiles; it += 2 * di) {
        step(qa, ga, DOUBLE ? qb : qa, DOUBLE ? gb : ga, it, 0);
        if (it + di < ntiles) step(DOUBLE ? qb : qa, DOUBLE ? gb : ga, qa, ga, it + di, DOUBLE ? 1 : 0);
    }

    if constexpr (SPLIT) {
        auto write = [&](const f32x16(&acc)[DT], void* to, float scale) {
            __syncthreads();
            Join<T, D>::keep(q_a, g_a, acc, lane, wave);
            __syncthreads();
            for (int i = threadIdx.x; i < 32 * (D / 4); i += kThreads) {
                const int r = i / (D / 4), d4 = i % (D / 4);
                if (row0 + r >= sp.lk) break;
                const f32x4 v = Join<T, D>::sum(q_a, g_a, r, d4, nullptr) * scale;
                const int64_t at = ((sp.k0 + row0 + r) * p.Hk + kvh) * D + 4 * d4;
                if (p.parts > 1) store4(static_cast<float*>(to) + part * p.total_k * p.Hk * D + at, v[0], v[1], v[2], v[3]);
                else store4(static_cast<T*>(to) + at, v[0], v[1], v[2], v[3]);
            }
        };
        write(dk, p.parts > 1 ? p.dkv_part : p.dk, p.scale);
        write(dv, p.parts > 1 ? p.dkv_part + p.parts * p.total_k * p.Hk * D : p.dv, 1.f);
        return;
    }
    T* dkg = static_cast<T*>(p.dk) + ((sp.k0 + key) * p.Hk + kvh) * D;
    T* dvg = static_cast<T*>(p.dv) + ((sp.k0 + key) * p.Hk + kvh) * D;
    if constexpr (PAIRED) {
        static_assert(!PAIRED || ELEMS * sizeof(T) == 32 * D * 4, "a tile's buffer holds one wave's sums");
        float* over = reinterpret_cast<float*>(wave == 0 ? q_a : wave == 1 ? g_a : wave == 2 ? q_b : g_b);
        auto merge = [&](f32x16(&acc)[DT], T* out, float f) {
            add_second(acc, over, n_own, lane);
            if (n_own == 0 && key < sp.lk) {
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int r = 0; r < 16; r += 8) store_rows(out + 32 * d, acc[d], r, half, f);
            }
        };
        merge(dk, dkg, p.scale);
        merge(dv, dvg, 1.f);
        return;
    }
    if (key >= sp.lk) return;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int r = 0; r < 16; r += 8) {
            store_rows(dkg + 32 * d, dk[d], r, half, p.scale);
            store_rows(dvg + 32 * d, dv[d], r, half, 1.f);
        }
}

// dk (blockIdx.y = 0) and dv (1) of one tile and key head from its parts, in order.
template <typename T, int D> __global__ void __launch_bounds__(kThreads) attn_parts_kernel(AttnParams p) {
    constexpr int OWN = kOwn<true>;
    int slot, kvh;
    work_item(blockIdx.x, p.k_slots, p.Hk, slot, kvh);
    const Span sp = find_span(p, slot, OWN, true);
    if (sp.tile < 0) return;
    const int64_t tensor = p.total_k * p.Hk * D;
    const float* from = p.dkv_part + blockIdx.y * p.parts * tensor;
    T* to = static_cast<T*>(blockIdx.y ? p.dv : p.dk);
    for (int i = threadIdx.x; i < OWN * (D / 4); i += kThreads) {
        const int r = sp.tile * OWN + i / (D / 4);
        if (r >= sp.lk) break;
        const int64_t at = ((sp.k0 + r) * p.Hk + kvh) * D + 4 * (i % (D / 4));
        f32x4 v{};
        for (int n = 0; n < p.parts; ++n) v += as_f32x4(ld16(from + n * tensor + at));
        store4(to + at, v[0], v[1], v[2], v[3]);
    }
}

// Bytes of LDS that a workgroup may have (160 KB), less the largest fixed part of a split kernel.
constexpr size_t kSplitBiasLds = 163840 - 139264;

template <typename T, int D, bool CAP, int BIAS, int SHARE>
int launch_dq(AttnParams p, hipStream_t stream) {
    constexpr int OWN = kOwn<SHARE == kSplit>;
    p.q_slots = (int)query_slots(p, OWN);
    set_each(p, OWN, 1);
    const int64_t grid = (int64_t)p.q_slots * (p.H / p.pack);
    const size_t lds = 4 * (size_t)bias_floats(BIAS, p.bk.max_distance, p.dtable != nullptr);
    if (BIAS == kBiasBuckets && hipFuncSetAttribute(reinterpret_cast<const void*>(&attn_dq_kernel<T, D, CAP, BIAS, SHARE>),
                                                    hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) != hipSuccess)
        return -1;
    if (grid > 0)
        hipLaunchKernelGGL((attn_dq_kernel<T, D, CAP, BIAS, SHARE>), dim3((unsigned)grid),
                           dim3(SHARE == kPaired ? 2 * kThreads : kThreads), lds, stream, p);
    if (p.dtable) hipLaunchKernelGGL(attn_dtable_kernel, dim3((unsigned)p.H), dim3(kThreads), 0, stream, p);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}
template <typename T, int D, bool CAP, int BIAS, int SHARE>
int launch_dkv(AttnParams p, hipStream_t stream) {
    constexpr int OWN = kOwn<SHARE == kSplit>;
    p.k_slots = (int)attn_slots(p.cu_k, p.total_k, p.nseq, OWN);
    set_each(p, 1, OWN);
    p.parts = SHARE == kSplit && p.dkv_part ? attn_key_parts(p.cu_k, p.total_k, p.nseq, p.Hk, Tile<T, D>::RB) : 1;
    const int64_t grid = (int64_t)p.k_slots * p.Hk * p.parts;
    const size_t lds = 4 * (size_t)bias_floats(BIAS, p.bk.max_distance, false) * (SHARE == kSplit ? p.H / p.Hk : 1);
    if (BIAS == kBiasBuckets && hipFuncSetAttribute(reinterpret_cast<const void*>(&attn_dkv_kernel<T, D, CAP, BIAS, SHARE>),
                                                    hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) != hipSuccess)
        return -1;
    if (grid > 0)
        hipLaunchKernelGGL((attn_dkv_kernel<T, D, CAP, BIAS, SHARE>), dim3((unsigned)grid),
                           dim3(SHARE == kPaired ? 2 * kThreads : kThreads), lds, stream, p);
    if (p.parts > 1)
        hipLaunchKernelGGL((attn_parts_kernel<T, D>), dim3((unsigned)(p.k_slots * p.Hk), 2), dim3(kThreads), 0, stream, p);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}
template <typename T, int D, bool CAP, int BIAS>
int launch_bwd(const AttnParams& p, hipStream_t stream) {
    // (a bias for every head of a group, or the sums by distance, may not fit beside a split kernel's tiles)
    const bool dq_fits = 4 * (size_t)bias_floats(BIAS, p.bk.max_distance, p.dtable != nullptr) <= kSplitBiasLds;
    const bool dkv_fits = 4 * (size_t)bias_floats(BIAS, p.bk.max_distance, false) * (p.H / p.Hk) <= kSplitBiasLds;
    AttnParams d = p;
    d.pack = query_pack(p, BIAS);
    const bool dq_split = dq_fits && query_slots(d, kOwn<false>) * (d.H / d.pack) < attn_split_below(Tile<T, D>::RB);
    const bool dkv_split = dkv_fits && attn_slots(p.cu_k, p.total_k, p.nseq, kOwn<false>) * p.Hk < attn_split_below(Tile<T, D>::RB);
    constexpr int WHOLE = sizeof(T) == 2 && D == 128 ? kPaired : kAlone, WHOLE_DQ = BIAS != kBiasBuckets ? WHOLE : kAlone;
    // (a split kernel has few workgroups)
    if ((!dq_split && !launchable(query_slots(d, kOwn<false>) * (d.H / d.pack), WHOLE_DQ == kPaired ? 2 * kThreads : kThreads)) ||
        (!dkv_split && !launchable(attn_slots(p.cu_k, p.total_k, p.nseq, kOwn<false>) * p.Hk, WHOLE == kPaired ? 2 * kThreads : kThreads)))
        return -2;
    d.plan_q = d.plan_k = nullptr;
    AttnParams with_plan = p;
    with_plan.pack = d.pack;
    if (p.plan_q && !(dq_split && dkv_split)) {
        // sequences of different lengths, and more than a round of workgroups: the longest first
        hipLaunchKernelGGL(attn_plan_kernel, dim3(2), dim3(kPlanThreads), 0, stream, with_plan, dq_split ? 0 : kOwn<false>, dkv_split ? 0 : kOwn<false>);
        if (!dq_split) d.plan_q = p.plan_q;
        if (!dkv_split) d.plan_k = p.plan_k;
    }
    int rc = dq_split ? launch_dq<T, D, CAP, BIAS, kSplit>(d, stream) : launch_dq<T, D, CAP, BIAS, WHOLE_DQ>(d, stream);
    if (rc == 0) rc = dkv_split ? launch_dkv<T, D, CAP, BIAS, kSplit>(d, stream) : launch_dkv<T, D, CAP, BIAS, WHOLE>(d, stream);
    return rc;
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

int launch_attn_backward(const AttnParams& p, int dtype, int D, int bias, hipStream_t stream) {
    return dtype == 1 ? attn::launch_bwd<__bf16>(p, D, bias, stream) : attn::launch_bwd<float>(p, D, bias, stream);
}

}  // namespace ssd
