// The paged cache in 8 bits, gfx950: the append that quantises, attention of one query per sequence over it, and the
// read-back.  Values stand for scale * x8, x8 an int8 or an e4m3 float, with a scale for each token and key head.
//
// kv8_decode_kernel is bound by the cache's bytes, each read once.  As attn_decode_kernel: a wave takes 32-key blocks of one
// (sequence, key head, split) in turn with a running maximum and sum of its own, for up to 16 query heads of the group (the
// columns of 16x16 MFMA tiles).  Either form of x8 is exact in bf16, so the products go through bf16 MFMAs on x8 itself: the
// key's scale is a factor of its score, the value's scale one of its weight.  fp32 queries and weights are taken in
// three bf16 terms, which together hold their 24 bits; the weights of a bf16 call in two (2^-16 of each), so that y is off by its own
// rounding: a weight has the value's scale in it and the divisor has not, so one term's roundings (up to 2^-8) would not drop out of
// a sum that one key dominates (errors of 2.4e-3 of y with one term, 1.66e-3 with two).
// 64 sequences of up to 8192 keys, 64/8 heads of 128, bf16 queries: 152 us and 5 for the join, 606 MB (4.0 TB/s; the same keys
// in bf16 250 us); 17 sequences of up to 4001 keys, 24 heads of 64, capped, biased by distance: 63 and 5 us.
// Of both types and forms, us, 64 sequences to 8192 keys, 64/8 heads of 32, 64, 128 (172, 326, 632 MB), and 17 sequences, 24 heads of 64, capped:
//     bf16  int8  82 111 171  62    e4m3  72 106 161  47         fp32  int8  92 132 217  75    e4m3  83 126 199  60
// fp32 queries' three terms are 48 registers at 128 wide; with int8's widening all but two of those kernels spill 19 to 27 of 256.
// Two waves a SIMD: four spill (much slower), and neither lanes in another order over a key's bytes nor non-temporal loads change it.
#include "ssd_attn_join.h"
#include "ssd_kv8_launch.h"
#include "ssd_rotary_common.h"

namespace ssd {
namespace attn {
namespace {

constexpr int kG = 16;      // query heads a workgroup takes
constexpr int kBlock = 32;  // keys of a block
enum { kInt8 = 0, kE4m3 = 1 };

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Eight held values as bf16 (exact).
template <int FORM> __device__ __forceinline__ bf16x8 widen(uint2 v) {
    const uint32_t w[2] = {v.x, v.y};
    bf16x8 f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (FORM == kE4m3) {
            const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.f, true);
            f[4 * i] = a[0];
            f[4 * i + 1] = a[1];
            f[4 * i + 2] = b[0];
            f[4 * i + 3] = b[1];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[4 * i + j] = (__bf16)(float)(int8_t)(w[i] >> (8 * j));
        }
    }
    return f;
}
template <int FORM> __device__ __forceinline__ float widen_one(uint8_t v) {
    if constexpr (FORM == kE4m3) return __builtin_amdgcn_cvt_f32_fp8((int)v, 0);
    else return (float)(int8_t)v;
}

template <typename T> constexpr int terms_of() { return sizeof(T) == 4 ? 3 : 1; }

// x as TERMS bf16 terms, each the rounded rest of those before it.
template <int TERMS> __device__ __forceinline__ void split(const float (&x)[8], bf16x8 (&f)[TERMS]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float rest = x[e];
#pragma unroll
        for (int u = 0; u < TERMS; ++u) {
            f[u][e] = (__bf16)rest;
            rest -= (float)f[u][e];
        }
    }
}

template <typename T, int D, int FORM, bool CAP, int BIAS, int NW>
__global__ void __launch_bounds__(NW * kWave, NW == kWaves ? 2 : 1) kv8_decode_kernel(DecodeParams p, Kv8Pages pages, int64_t units) {
    constexpr int TERMS = terms_of<T>(), WTERMS = TERMS > 2 ? TERMS : 2;  // of the queries, of the weights
    constexpr int NT = D / 32, DT = D / 16;
    constexpr int KB = D >= 64 ? 16 : 8;      // bytes of a key's load: lane group g has KB g .. of each 4 KB
    constexpr int NK = D / (4 * KB);          // loads of a key
    constexpr int CH = D / 16;                // 16-byte chunks of a value
    constexpr int VL = kBlock * CH / kWave;   // of them, those a lane stages
    constexpr int VS = D + 8;                 // LDS row stride of V, bf16
    constexpr int kTile = kBlock * VS * 2, kJoin = kG * D * 4;  // (a wave's O for the join takes the same memory)
    __shared__ __attribute__((aligned(16))) char vmem[NW][kTile > kJoin ? kTile : kJoin];
    __shared__ __attribute__((aligned(16))) float scales[NW][2 * kBlock];
    __shared__ float stat[NW][2][kG];
    extern __shared__ float extra[];          // buckets: [total][kG] bias, then bucket by distance

    // the key heads and tiles of one (sequence, split) share lines of the scales and of the block table: one XCD has them
    const int group = p.H / p.Hk, tiles = (group + kG - 1) / kG, mates = p.Hk * tiles;
    const uint32_t turn = blockIdx.x / 8;
    const int64_t unit = (int64_t)(turn / mates) * 8 + blockIdx.x % 8;
    if (unit >= units) return;
    const int tile = turn % mates % tiles, kvh = turn % mates / tiles, split_id = (int)(unit % p.splits), s = (int)(unit / p.splits);
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, col = lane % 16, g = lane / 16;
    const int heads = min(kG, group - tile * kG), head0 = kvh * group + tile * kG;
    const int len = (int)clamp64(p.seq_lens[s], 0, (int64_t)p.max_pages * p.page_size);
    const int blocks = (len + kBlock - 1) / kBlock, per = (blocks + p.splits - 1) / p.splits;
    const int b0 = split_id * per, b1 = min(b0 + per, blocks);

    Score sc;
    sc.init<T>(fabsf(p.scale), p.cap, CAP);
    const int head = head0 + min(col, heads - 1);
    bf16x8 qf[NT][TERMS];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        // (the order of a key's loads: the first and second half of a lane's 16 bytes are two steps)
        const int d = KB == 16 ? 64 * (t / 2) + 16 * g + 8 * (t % 2) : 8 * g;
        const T* q = static_cast<const T*>(p.q) + (int64_t)s * p.q_stride + (int64_t)head * D + d;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = p.scale < 0.f ? -to_f32(q[e]) : to_f32(q[e]);
        split<TERMS>(x, qf[t]);
    }
    float slope2 = 0.f, far = 0.f;
    const int md = p.bk.max_distance;
    const float* bias = extra;
    const int* bucket = reinterpret_cast<const int*>(extra + p.bk.total * kG);
    if constexpr (BIAS == kBiasSlopes) slope2 = p.slopes[head] * kLog2e;
    if constexpr (BIAS == kBiasBuckets) {
        for (int i = threadIdx.x; i < p.bk.total * kG; i += NW * kWave)
            extra[i] = p.table[(int64_t)(i / kG) * p.H + head0 + min(i % kG, heads - 1)] * kLog2e;
        for (int i = threadIdx.x; i <= md; i += NW * kWave) reinterpret_cast<int*>(extra + p.bk.total * kG)[i] = bucket_of(p.bk, -i) * kG;
        __syncthreads();
        far = bias[bucket[md] + col];
    }

    __bf16* vt = reinterpret_cast<__bf16*>(vmem[wave]);
    const int64_t row = (int64_t)p.Hk * D;  // from one key of a page to the next

    f32x4 o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = f32x4{};
    float m = kNoMax, l = 0.f;

    typedef uint32_t key_load __attribute__((ext_vector_type(KB / 4)));
    key_load kb[2][NK];
    uint4 vb[VL];
    float sb = 0.f;  // lanes 0 .. 31: the scales of the block's keys, 32 .. 63: of its values
    int ok = 0;      // bit n: the block's 16 keys 16 n .. are on a page
    auto fetch = [&](int b) {
        ok = 0;
        int64_t first[2];
        int have[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int key0 = b * kBlock + 16 * n;
            int page = -1;
            if (key0 < len) {
                page = __builtin_amdgcn_readfirstlane(p.block_table[(int64_t)s * p.max_pages + key0 / p.page_size]);
                page = page >= 0 && page < p.num_pages ? page : -1;
            }
            if (page >= 0) ok |= 1 << n;
            // keys past the length, and keys of no page, are not read: zeros stand for them
            first[n] = ((int64_t)(page < 0 ? 0 : page) * p.page_size + key0 % p.page_size) * p.Hk + kvh;
            have[n] = page < 0 ? 0 : len - key0;
            const uint8_t* kp = pages.k + first[n] * D + (int64_t)col * row + g * KB;
#pragma unroll
            for (int t = 0; t < NK; ++t) kb[n][t] = col < have[n] ? *reinterpret_cast<const key_load*>(kp + 4 * KB * t) : key_load{};
        }
#pragma unroll
        for (int i = 0; i < VL; ++i) {
            const int idx = lane + kWave * i, r = idx / CH, n = r / 16;
            vb[i] = r % 16 < have[n] ? ld16(pages.v + first[n] * D + (int64_t)(r % 16) * row + (idx % CH) * 16) : uint4{};
        }
        const int n = lane / 16 % 2;
        const float* sp = (lane < 32 ? pages.k_scale : pages.v_scale) + first[n] + (int64_t)col * p.Hk;
        sb = col < have[n] ? *sp : 0.f;
    };
    int b = b0 + wave;
    if (b < b1) fetch(b);
    for (; b < b1; b += NW) {
        bf16x8 kf[2][NT];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const key_load x = kb[n][t / (KB / 8)];
                kf[n][t] = widen<FORM>(uint2{x[KB == 16 ? 2 * (t % 2) : 0], x[KB == 16 ? 2 * (t % 2) + 1 : 1]});
            }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < VL; ++i) {
            const int idx = lane + kWave * i, r = idx / CH;
            __bf16* to = vt + r * VS + (idx % CH) * 16;
            st16(to, __builtin_bit_cast(uint4, widen<FORM>(uint2{vb[i].x, vb[i].y})));
            st16(to + 8, __builtin_bit_cast(uint4, widen<FORM>(uint2{vb[i].z, vb[i].w})));
        }
        scales[wave][lane] = sb;
        __builtin_amdgcn_wave_barrier();
        const int here = ok;
        if (b + NW < b1) fetch(b + NW);
        f32x4 sv[2], vs[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            sv[n] = f32x4{};
#pragma unroll
            for (int u = TERMS - 1; u >= 0; --u)
#pragma unroll
                for (int t = 0; t < NT; ++t) sv[n] = mfma_bf16(kf[n][t], qf[t][u], sv[n]);
            sv[n] *= *reinterpret_cast<const f32x4*>(&scales[wave][16 * n + 4 * g]);
            vs[n] = *reinterpret_cast<const f32x4*>(&scales[wave][kBlock + 16 * n + 4 * g]);
        }
        // register r of tile n: key b * 32 + 16 n + 4 g + r of query head `col`
        const int key0 = b * kBlock + 4 * g;
        const bool all_far = len - 1 - (b * kBlock + kBlock - 1) >= md;
        float mx = -INFINITY;
        if constexpr (CAP) sc.template capped<T>(sv);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int key = key0 + 16 * n + r;
                float x = CAP ? sv[n][r] : sv[n][r] * sc.a;
                if constexpr (BIAS == kBiasSlopes) x -= slope2 * (float)(len - 1 - key);
                if constexpr (BIAS == kBiasBuckets) x += all_far ? far : bias[bucket[min(max(len - 1 - key, 0), md)] + col];
                x = key < len && (here >> n & 1) ? x : -INFINITY;
                sv[n][r] = x;
                mx = fmaxf(mx, x);
            }
        mx = fmaxf(mx, __shfl_xor(mx, 16, kWave));
        mx = fmaxf(mx, __shfl_xor(mx, 32, kWave));
        if (__any(mx > m)) {
            const float next = fmaxf(m, mx), keep = exp2_hw(m - next);
            m = next;
            l *= keep;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d] *= keep;
        }
        // weights with the values' scales, contracting over the 32 keys in the row order of the two stacked tiles
        float w[8];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float e = exp2_hw(sv[n][r] - m);
                l += e;
                w[4 * n + r] = e * vs[n][r];
            }
        bf16x8 pf[WTERMS];
        split<WTERMS>(w, pf);
        const __bf16* at = vt + (4 * g + col / 4) * VS + 4 * (col % 4);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(at + 16 * d));
            const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(at + 16 * VS + 16 * d));
            const v8i16 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
            for (int u = WTERMS - 1; u >= 0; --u) o[d] = mfma_bf16(__builtin_bit_cast(bf16x8, v), pf[u], o[d]);
        }
    }

    // the waves' shares: O^T register r of tile d is column `col`, row 16 d + 4 g + r
    l += __shfl_xor(l, 16, kWave);
    l += __shfl_xor(l, 32, kWave);
    if (g == 0) {
        stat[wave][0][col] = m;
        stat[wave][1][col] = l;
    }
    float* mine = reinterpret_cast<float*>(vmem[wave]) + col * D + 4 * g;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int d = 0; d < DT; ++d) st16(mine + 16 * d, __builtin_bit_cast(uint4, o[d]));
    __syncthreads();
    for (int i = threadIdx.x; i < heads * (D / 4); i += NW * kWave) {
        const int c = i / (D / 4), d = 4 * (i % (D / 4));
        float top = stat[0][0][c];
#pragma unroll
        for (int w = 1; w < NW; ++w) top = fmaxf(top, stat[w][0][c]);
        float sum = 0.f;
        f32x4 v{};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = exp2_hw(stat[w][0][c] - top);
            sum += f * stat[w][1][c];
            v += f * *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(vmem[w]) + c * D + d);
        }
        const int64_t at = (int64_t)s * p.H + head0 + c;
        if (p.splits == 1) {
            const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
            store4(static_cast<T*>(p.y) + at * D + d, v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
        } else {
            st16(p.part_o + (at * p.splits + split_id) * D + d, __builtin_bit_cast(uint4, v));
            if (d == 0) {
                p.part_ml[(at * p.splits + split_id) * 2] = top;
                p.part_ml[(at * p.splits + split_id) * 2 + 1] = sum;
            }
        }
    }
}

template <typename T, int D, int FORM, bool CAP, int BIAS, int NW>
int launch_decode(const DecodeParams& p, const Kv8Pages& pages, hipStream_t stream) {
    const int64_t group = p.H / p.Hk, units = p.nseq * p.splits, grid = (units + 7) / 8 * 8 * p.Hk * ((group + kG - 1) / kG);
    if (!launchable(grid, NW * kWave)) return -2;
    const size_t lds = BIAS == kBiasBuckets ? 4 * (size_t)(p.bk.total * kG + p.bk.max_distance + 1) : 0;
    const auto kernel = &kv8_decode_kernel<T, D, FORM, CAP, BIAS, NW>;
    if (lds > 0 && hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) != hipSuccess)
        return -1;
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(NW * kWave), lds, stream, p, pages, units);
    if (hipGetLastError() != hipSuccess) return -1;
    return p.splits > 1 ? launch_join<T, D>(p, stream) : 0;
}
template <typename T, int D, int FORM, bool CAP, int BIAS>
int launch_decode(const DecodeParams& p, const Kv8Pages& pages, hipStream_t stream) {
    return p.wide ? launch_decode<T, D, FORM, CAP, BIAS, 2 * kWaves>(p, pages, stream) : launch_decode<T, D, FORM, CAP, BIAS, kWaves>(p, pages, stream);
}
template <typename T, int D, int FORM>
int launch_decode(const DecodeParams& p, const Kv8Pages& pages, int bias, hipStream_t stream) {
    const bool cap = p.cap > 0.f;
    switch (bias) {
        case kBiasNone:
            return cap ? launch_decode<T, D, FORM, true, kBiasNone>(p, pages, stream) : launch_decode<T, D, FORM, false, kBiasNone>(p, pages, stream);
        case kBiasSlopes:
            return cap ? launch_decode<T, D, FORM, true, kBiasSlopes>(p, pages, stream) : launch_decode<T, D, FORM, false, kBiasSlopes>(p, pages, stream);
        default:
            return cap ? launch_decode<T, D, FORM, true, kBiasBuckets>(p, pages, stream) : launch_decode<T, D, FORM, false, kBiasBuckets>(p, pages, stream);
    }
}
template <typename T, int FORM>
int launch_decode(const DecodeParams& p, const Kv8Pages& pages, int D, int bias, hipStream_t stream) {
    switch (D) {
        case 32: return launch_decode<T, 32, FORM>(p, pages, bias, stream);
        case 64: return launch_decode<T, 64, FORM>(p, pages, bias, stream);
        case 128: return launch_decode<T, 128, FORM>(p, pages, bias, stream);
        default: return -2;
    }
}

// One token a workgroup: its queries and keys rotated, its keys and values quantised.  A head is D / E neighbouring lanes
// (16 bytes of input each), whose largest magnitude is taken by shuffles.  Rotated keys are not rounded before they are
// quantised: the sines and cosines come from fp64, each product is rounded by itself, and the division is the exact one, so
// that the held value is that of the formula.  (Their largest magnitude as bits: NaN and infinities are above all else.)
// Bound by bytes: 16385 tokens, 32/8 heads of 128, bf16: 72 us, 5.1 TB/s.
template <typename T, int FORM>
__global__ void __launch_bounds__(kThreads) kv8_append_kernel(AppendParams p, Kv8Pages pages) {
    constexpr int E = 16 / (int)sizeof(T);
    typedef T vec __attribute__((ext_vector_type(E)));
    __shared__ float cs[kMaxRot], sn[kMaxRot];
    const int64_t tok = (int64_t)blockIdx.y * kTokenRow + blockIdx.x;
    if (tok >= p.tokens) return;
    int64_t s = tok, end = tok + 1;
    if (p.cu) {
        s = last_at_most((int)p.nseq, [&](int i) { return p.cu[i] <= tok; });
        end = p.cu[s + 1];
        if (tok < p.cu[s] || tok >= end) return;  // a token of no sequence
    }
    const int64_t pos = p.seq_lens[s] - (end - tok);
    for (int i = threadIdx.x; i < p.rot; i += kThreads) {
        double a, b;
        sincospi(half_turns(pos, p.inv_freq[i]), &a, &b);
        cs[i] = (float)b;
        sn[i] = (float)a;
    }
    int64_t slot = -1;
    if (pos >= 0 && pos < (int64_t)p.max_pages * p.page_size) {
        const int page = p.block_table[s * p.max_pages + pos / p.page_size];
        if (page >= 0 && page < p.num_pages) slot = (int64_t)page * p.page_size + pos % p.page_size;
    }
    __syncthreads();
    const int D = p.D, CH = D / E, qc = p.q ? p.H * CH : 0, kc = p.Hk * CH;
    const int total = slot >= 0 ? qc + 2 * kc : qc;
    for (int i = threadIdx.x; i < total; i += kThreads) {
        const int which = i < qc ? 0 : i < qc + kc ? 1 : 2, at = which == 0 ? i : which == 1 ? i - qc : i - qc - kc, d = (at % CH) * E;
        const T* in = which == 0   ? static_cast<const T*>(p.q) + tok * p.q_stride
                      : which == 1 ? static_cast<const T*>(p.k) + tok * p.k_stride
                                   : static_cast<const T*>(p.v) + tok * p.v_stride;
        const vec x = __builtin_bit_cast(vec, ld16(in + at * E));
        float y[E];
        if (which < 2 && d < 2 * p.rot) {
            const int over = p.interleaved ? 0 : d < p.rot ? p.rot : -p.rot;
            const vec z = __builtin_bit_cast(vec, ld16(in + at * E + over));
            rotate<T, E>(x, z, d, p.rot, p.interleaved, cs, sn, y);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) y[e] = (float)x[e];
        }
        if (which == 0) {
            vec out;
#pragma unroll
            for (int e = 0; e < E; ++e) out[e] = (T)y[e];
            st16(static_cast<T*>(p.q_out) + tok * p.H * D + at * E, __builtin_bit_cast(uint4, out));
            continue;
        }
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) top = max(top, __builtin_bit_cast(uint32_t, y[e]) & 0x7fffffffu);
        for (int off = 1; off < CH; off <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, kWave));
        constexpr float kTop = FORM == kE4m3 ? 448.f : 127.f;
        const bool finite = top < 0x7f800000u;
        const float largest = __builtin_bit_cast(float, top);
        float scale = finite ? largest * (1.f / kTop) : NAN;
        // (a subnormal scale has few bits: it is rounded up, or the largest value would not fit)
        if (scale < 0x1p-126f && scale * kTop < largest) scale = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, scale) + 1);
        const float by = scale > 0.f ? scale : 1.f;
        uint32_t out[E / 4];
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            float r[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = finite ? fminf(fmaxf(y[e + j] / by, -kTop), kTop) : 0.f;
            if constexpr (FORM == kE4m3) {
                int v = __builtin_amdgcn_cvt_pk_fp8_f32(r[0], r[1], 0, false);
                out[e / 4] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(r[2], r[3], v, true);
            } else {
                uint32_t v = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) v |= ((uint32_t)(int)rintf(r[j]) & 0xffu) << (8 * j);
                out[e / 4] = v;
            }
        }
        uint8_t* to = (which == 1 ? pages.k : pages.v) + slot * p.Hk * D + at * E;
        if constexpr (E == 8) *reinterpret_cast<uint2*>(to) = uint2{out[0], out[E / 4 - 1]};
        else *reinterpret_cast<uint32_t*>(to) = out[0];
        if (d == 0) (which == 1 ? pages.k_scale : pages.v_scale)[slot * p.Hk + at / CH] = scale;
    }
}

// One row of the output for each wave.  Bound by the bytes that it writes: nine sequences of up to 4001 tokens, 8 heads of 128, to bf16: 27 us.
template <typename T, int FORM>
__global__ void __launch_bounds__(kThreads) kv8_read_kernel(Kv8ReadParams p) {
    const int64_t tok = ((int64_t)blockIdx.y * kTokenRow + blockIdx.x) * kWaves + threadIdx.x / kWave;
    if (tok >= p.tokens) return;
    int64_t s, first;
    if (p.cu) {
        s = last_at_most((int)p.nseq, [&](int i) { return p.cu[i] <= tok; });
        first = p.cu[s];
        if (tok < first || tok >= p.cu[s + 1]) return;  // a row of no sequence
    } else {
        s = tok / p.each;
        first = s * p.each;
    }
    const int64_t pos = tok - first;
    int64_t slot = -1;
    if (pos < p.seq_lens[s] && pos < (int64_t)p.max_pages * p.page_size) {
        const int page = p.block_table[s * p.max_pages + pos / p.page_size];
        if (page >= 0 && page < p.num_pages) slot = (int64_t)page * p.page_size + pos % p.page_size;
    }
    const int row = p.Hk * p.D, n = row / 8;
    for (int i = threadIdx.x % kWave; i < 2 * n; i += kWave) {
        const bool key = i < n;
        const int at = 8 * (key ? i : i - n);
        T* out = static_cast<T*>(key ? p.k : p.v) + tok * row + at;
        float y[8] = {};
        if (slot >= 0) {
            const uint2 x = ld8((key ? p.pages.k : p.pages.v) + slot * row + at);
            const float scale = (key ? p.pages.k_scale : p.pages.v_scale)[slot * p.Hk + at / p.D];
            const bf16x8 f = widen<FORM>(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = (float)f[e] * scale;
        }
        store4(out, y[0], y[1], y[2], y[3]);
        store4(out + 4, y[4], y[5], y[6], y[7]);
    }
}

}  // namespace
}  // namespace attn

int launch_kv8_decode(const DecodeParams& p, const Kv8Pages& pages, int dtype, int format, int D, int bias, hipStream_t stream) {
    using namespace attn;
    if (dtype == 1) return format == kE4m3 ? launch_decode<__bf16, kE4m3>(p, pages, D, bias, stream) : launch_decode<__bf16, kInt8>(p, pages, D, bias, stream);
    return format == kE4m3 ? launch_decode<float, kE4m3>(p, pages, D, bias, stream) : launch_decode<float, kInt8>(p, pages, D, bias, stream);
}

int launch_kv8_append(const AppendParams& p, const Kv8Pages& pages, int dtype, int format, hipStream_t stream) {
    using namespace attn;
    const auto kernel = dtype == 1 ? (format == kE4m3 ? &kv8_append_kernel<__bf16, kE4m3> : &kv8_append_kernel<__bf16, kInt8>)
                                   : (format == kE4m3 ? &kv8_append_kernel<float, kE4m3> : &kv8_append_kernel<float, kInt8>);
    hipLaunchKernelGGL(kernel, token_grid(p.tokens), dim3(kThreads), 0, stream, p, pages);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_kv8_read(const Kv8ReadParams& p, int dtype, int format, hipStream_t stream) {
    using namespace attn;
    const auto kernel = dtype == 1 ? (format == kE4m3 ? &kv8_read_kernel<__bf16, kE4m3> : &kv8_read_kernel<__bf16, kInt8>)
                                   : (format == kE4m3 ? &kv8_read_kernel<float, kE4m3> : &kv8_read_kernel<float, kInt8>);
    hipLaunchKernelGGL(kernel, token_grid((p.tokens + kWaves - 1) / kWaves), dim3(kThreads), 0, stream, p);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace ssd
