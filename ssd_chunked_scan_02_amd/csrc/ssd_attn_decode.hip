// Attention of one query per sequence over a paged cache, and the append to that cache, gfx950.
//
// attn_decode_kernel reads every visible key and value once, which bounds it: 4 waves of a workgroup take
// the 32-key blocks of one (sequence, key head, split) in turn, each with a running maximum and sum of
// its own, for up to 16 query heads of the group at once (the column index of 16x16 MFMA tiles, so a
// group costs no more reads than one head).  S^T = K Q^T takes the keys straight from memory (a lane's
// 16 bytes of a key are an operand), P^T in its accumulator layout is the operand of O^T += V^T P^T, and
// the values go through a wave's own LDS to be read transposed.  A wave's next block is on its way while
// it works on the present one.  Few sequences are split along their keys so that the chip is filled; the
// splits' (m, l, O) are joined by attn_join_kernel.  The split of a sequence follows its length on the
// device, so a captured graph stays balanced as the cache grows.
//
// Measured: 64 sequences of up to 8192 keys, 64/8 heads of 128, bf16: 246 us and 4 for the join, 4.8 TB/s
// (a large copy reaches 5.1); 17 sequences of up to 4001 keys, 24 heads of 64, fp32: 111 us, 4.6 TB/s.  In fp32 at 128 wide
// the two blocks that a wave holds are 15 to 21 registers too many, which it spills: 62 sequences of 1000 keys, 8 key heads:
// 126 us, 4.0 TB/s.
//
// kv_append_kernel copies one token's keys and values into its page, rotated: bound by memory (16385 tokens, 32/8 heads
// of 128: 81 us, 5.0 TB/s), and for a decode step by its launch (64 tokens: 6 us).
#include "ssd_attn_common.h"
#include "ssd_attn_join.h"

namespace ssd {
namespace attn {
namespace {

constexpr int kG = 16;        // query heads a workgroup takes
constexpr int kBlock = 32;    // keys of a block

template <typename T> struct Op16;  // 16x16 tiles
template <> struct Op16<__bf16> {
    using Frag = bf16x8;
    static constexpr int kE = 8, kK = 32;
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) { return mfma_bf16(a, b, c); }
};
template <> struct Op16<float> {
    using Frag = f32x4;
    static constexpr int kE = 4, kK = 16;
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c = mfma_f32(a[i], b[i], c);
        return c;
    }
};

// Page of sequence s's 16 keys from `key` on; negative when it is none of the cache's pages.
__device__ __forceinline__ int page_of(const DecodeParams& p, int64_t s, int key) {
    const int page = p.block_table[s * p.max_pages + key / p.page_size];
    return page >= 0 && page < p.num_pages ? page : -1;
}

template <typename T, int D, bool CAP, int BIAS, int NW>
__global__ void __launch_bounds__(NW * kWave, NW == kWaves ? 2 : 1) attn_decode_kernel(DecodeParams p) {
    using O = Op16<T>;
    using Frag = typename O::Frag;
    constexpr int E = O::kE, NT = D / O::kK, DT = D / 16, CH = D / E;
    constexpr int VL = kBlock * CH / kWave;   // 16-byte chunks of V a lane stages
    constexpr int VS = D + E;                 // LDS row stride of V
    constexpr int kTile = kBlock * VS * (int)sizeof(T);
    constexpr int kJoin = kG * D * 4;         // a wave's O for the join, in the same memory
    __shared__ __attribute__((aligned(16))) char vmem[NW][kTile > kJoin ? kTile : kJoin];
    __shared__ float stat[NW][2][kG];
    extern __shared__ float extra[];          // buckets: [total][kG] bias, then bucket by distance

    const int group = p.H / p.Hk, tiles = (group + kG - 1) / kG;
    int id = blockIdx.x;
    const int split = id % p.splits;
    id /= p.splits;
    const int tile = id % tiles;
    id /= tiles;
    const int kvh = id % p.Hk, s = id / p.Hk;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, col = lane % 16, g = lane / 16;
    const int heads = min(kG, group - tile * kG), head0 = kvh * group + tile * kG;
    const int len = (int)clamp64(p.seq_lens[s], 0, (int64_t)p.max_pages * p.page_size);
    const int blocks = (len + kBlock - 1) / kBlock, per = (blocks + p.splits - 1) / p.splits;
    const int b0 = split * per, b1 = min(b0 + per, blocks);

    Score sc;
    sc.init<T>(fabsf(p.scale), p.cap, CAP);
    const int head = head0 + min(col, heads - 1);
    Frag qf[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
        qf[t] = signed_frag<T>(static_cast<const T*>(p.q) + (int64_t)s * p.q_stride + (int64_t)head * D + t * O::kK + g * E, p.scale);
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

    const T* kc = static_cast<const T*>(p.k_cache) + (int64_t)kvh * D;
    const T* vc = static_cast<const T*>(p.v_cache) + (int64_t)kvh * D;
    T* vt = reinterpret_cast<T*>(vmem[wave]);
    const int64_t row = (int64_t)p.Hk * D;  // from one key of a page to the next

    f32x4 o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = f32x4{};
    // (in bf16 the sum of the rounded weights, the divisor that takes out what their rounding has in common)
    float m = kNoMax, l = 0.f;

    uint4 kb[2][NT], vb[VL];
    int ok = 0;  // bit n: the block's 16 keys 16 n .. are on a page
    auto fetch = [&](int b) {
        ok = 0;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int key0 = b * kBlock + 16 * n;
            const int page = key0 < len ? __builtin_amdgcn_readfirstlane(page_of(p, s, key0)) : -1;
            if (page >= 0) ok |= 1 << n;
            // keys past the length, and keys of no page, are not read: zeros stand for them
            const int64_t first = ((int64_t)(page < 0 ? 0 : page) * p.page_size + key0 % p.page_size) * row;
            const int have = page < 0 ? 0 : len - key0;
            const T* kp = kc + first + (int64_t)col * row + g * E;
#pragma unroll
            for (int t = 0; t < NT; ++t) kb[n][t] = col < have ? ld16(kp + t * O::kK) : uint4{};
#pragma unroll
            for (int i = 0; i < VL / 2; ++i) {
                const int idx = lane + kWave * i, r = idx / CH;
                vb[n * (VL / 2) + i] = r < have ? ld16(vc + first + (int64_t)r * row + (idx % CH) * E) : uint4{};
            }
        }
    };
    int b = b0 + wave;
    if (b < b1) fetch(b);
    for (; b < b1; b += NW) {
        Frag kf[2][NT];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int t = 0; t < NT; ++t) kf[n][t] = __builtin_bit_cast(Frag, kb[n][t]);
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < VL; ++i) {
            const int idx = lane + kWave * (i % (VL / 2)), r = 16 * (i / (VL / 2)) + idx / CH;
            st16(vt + r * VS + (idx % CH) * E, vb[i]);
        }
        __builtin_amdgcn_wave_barrier();
        const int here = ok;
        f32x4 sv[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            sv[n] = f32x4{};
#pragma unroll
            for (int t = 0; t < NT; ++t) sv[n] = O::mma(kf[n][t], qf[t], sv[n]);
        }
        if (b + NW < b1) fetch(b + NW);
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
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                sv[n][r] = exp2_hw(sv[n][r] - m);
                if constexpr (sizeof(T) == 4) l += sv[n][r];
            }
        if constexpr (sizeof(T) == 2) {
            // contraction over the 32 keys in the row order of the two stacked tiles: 4 g + j, 16 + 4 g + j - 4
            bf16x8 pf;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                pf[j] = (__bf16)sv[0][j];
                pf[4 + j] = (__bf16)sv[1][j];
            }
            l = sum_of(pf, l);
            const __bf16* at = reinterpret_cast<const __bf16*>(vt) + (4 * g + col / 4) * VS + 4 * (col % 4);
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(at + 16 * d));
                const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(at + 16 * VS + 16 * d));
                const v8i16 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                o[d] = mfma_bf16(__builtin_bit_cast(bf16x8, v), pf, o[d]);
            }
        } else {
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        o[d] = mfma_f32(reinterpret_cast<const float*>(vt)[(16 * n + 4 * g + r) * VS + 16 * d + col], sv[n][r], o[d]);
        }
    }

    // the four waves' shares: O^T register r of tile d is column `col`, row 16 d + 4 g + r
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
            st16(p.part_o + (at * p.splits + split) * D + d, __builtin_bit_cast(uint4, v));
            if (d == 0) {
                p.part_ml[(at * p.splits + split) * 2] = top;
                p.part_ml[(at * p.splits + split) * 2 + 1] = sum;
            }
        }
    }
}

template <typename T, int D, bool CAP, int BIAS, int NW>
int launch_decode(const DecodeParams& p, hipStream_t stream) {
    const int64_t group = p.H / p.Hk, grid = p.nseq * p.Hk * ((group + kG - 1) / kG) * p.splits;
    if (!launchable(grid, NW * kWave)) return -2;
    const size_t lds = BIAS == kBiasBuckets ? 4 * (size_t)(p.bk.total * kG + p.bk.max_distance + 1) : 0;
    if (lds > 0 && hipFuncSetAttribute(reinterpret_cast<const void*>(&attn_decode_kernel<T, D, CAP, BIAS, NW>),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) != hipSuccess)
        return -1;
    hipLaunchKernelGGL((attn_decode_kernel<T, D, CAP, BIAS, NW>), dim3((unsigned)grid), dim3(NW * kWave), lds, stream, p);
    if (hipGetLastError() != hipSuccess) return -1;
    return p.splits > 1 ? launch_join<T, D>(p, stream) : 0;
}
template <typename T, int D, bool CAP, int BIAS>
int launch_decode(const DecodeParams& p, hipStream_t stream) {
    return p.wide ? launch_decode<T, D, CAP, BIAS, 2 * kWaves>(p, stream) : launch_decode<T, D, CAP, BIAS, kWaves>(p, stream);
}
template <typename T, int D, bool CAP>
int launch_decode(const DecodeParams& p, int bias, hipStream_t stream) {
    switch (bias) {
        case kBiasNone: return launch_decode<T, D, CAP, kBiasNone>(p, stream);
        case kBiasSlopes: return launch_decode<T, D, CAP, kBiasSlopes>(p, stream);
        default: return launch_decode<T, D, CAP, kBiasBuckets>(p, stream);
    }
}
template <typename T>
int launch_decode(const DecodeParams& p, int D, int bias, hipStream_t stream) {
    const bool cap = p.cap > 0.f;
    switch (D) {
        case 32: return cap ? launch_decode<T, 32, true>(p, bias, stream) : launch_decode<T, 32, false>(p, bias, stream);
        case 64: return cap ? launch_decode<T, 64, true>(p, bias, stream) : launch_decode<T, 64, false>(p, bias, stream);
        case 128: return cap ? launch_decode<T, 128, true>(p, bias, stream) : launch_decode<T, 128, false>(p, bias, stream);
        default: return -2;
    }
}

// One token a workgroup.  Its angles, pos * inv_freq in turns, are reduced in fp64 (pos * inv_freq is exact
// to 53 bits there, and a far position's turns leave an fp32 no fraction), their sine and cosine taken in
// fp32 once for all heads.  More tokens than a row of the grid holds go on in its next row (a loop over them
// instead: 100 us against 82 for 16385 tokens, 32/8 heads of 128).
constexpr int kAppendRow = 1 << 22;
template <typename T>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(AppendParams p) {
    constexpr int E = 16 / (int)sizeof(T);
    __shared__ float cs[2][kMaxRot];
    const int64_t tok = (int64_t)blockIdx.y * kAppendRow + blockIdx.x;
    if (tok >= p.tokens) return;
    int64_t s = tok, end = tok + 1;
    if (p.cu) {
        s = last_at_most((int)p.nseq, [&](int i) { return p.cu[i] <= tok; });
        end = p.cu[s + 1];
        if (tok < p.cu[s] || tok >= end) return;  // a token of no sequence
    }
    const int64_t pos = p.seq_lens[s] - (end - tok);
    for (int i = threadIdx.x; i < p.rot; i += kThreads) {
        const double turns = (double)pos * (double)p.inv_freq[i] * 0.15915494309189535;
        float sn, cn;
        sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cn);
        cs[0][i] = cn;
        cs[1][i] = sn;
    }
    int64_t slot = -1;
    if (pos >= 0 && pos < (int64_t)p.max_pages * p.page_size) {
        const int page = p.block_table[s * p.max_pages + pos / p.page_size];
        if (page >= 0 && page < p.num_pages) slot = (int64_t)page * p.page_size + pos % p.page_size;
    }
    __syncthreads();
    const int D = p.D, CH = D / E, qc = p.q ? p.H * CH : 0, kc = p.Hk * CH;
    const int total = slot >= 0 ? qc + 2 * kc : qc;
    typedef T vec __attribute__((ext_vector_type(E)));
    for (int i = threadIdx.x; i < total; i += kThreads) {
        const T* in;
        T* out;
        int at;
        if (i < qc) {
            in = static_cast<const T*>(p.q) + tok * p.q_stride;
            out = static_cast<T*>(p.q_out) + tok * p.H * D;
            at = i;
        } else if (i < qc + kc) {
            in = static_cast<const T*>(p.k) + tok * p.k_stride;
            out = static_cast<T*>(p.k_cache) + slot * p.Hk * D;
            at = i - qc;
        } else {
            in = static_cast<const T*>(p.v) + tok * p.v_stride;
            out = static_cast<T*>(p.v_cache) + slot * p.Hk * D;
            at = i - qc - kc;
        }
        const vec x = __builtin_bit_cast(vec, ld16(in + at * E));
        const int d = (at % CH) * E;  // first element within its head
        if (i >= qc + kc || d >= 2 * p.rot) {
            st16(out + at * E, __builtin_bit_cast(uint4, x));
            continue;
        }
        vec y;
        if (p.interleaved) {
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float c = cs[0][(d + e) / 2], sn = cs[1][(d + e) / 2], a = (float)x[e], b = (float)x[e + 1];
                y[e] = (T)(a * c - b * sn);
                y[e + 1] = (T)(b * c + a * sn);
            }
        } else {
            const bool low = d < p.rot;
            const vec z = __builtin_bit_cast(vec, ld16(in + at * E + (low ? p.rot : -p.rot)));
            const int f = low ? d : d - p.rot;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float c = cs[0][f + e], sn = cs[1][f + e];
                y[e] = (T)((float)x[e] * c + (low ? -(float)z[e] : (float)z[e]) * sn);
            }
        }
        st16(out + at * E, __builtin_bit_cast(uint4, y));
    }
}

}  // namespace
}  // namespace attn

int launch_attn_decode(const DecodeParams& p, int dtype, int D, int bias, hipStream_t stream) {
    return dtype == 1 ? attn::launch_decode<__bf16>(p, D, bias, stream) : attn::launch_decode<float>(p, D, bias, stream);
}

int launch_kv_append(const AppendParams& p, int dtype, hipStream_t stream) {
    const dim3 grid((unsigned)(p.tokens < attn::kAppendRow ? p.tokens : attn::kAppendRow),
                    (unsigned)((p.tokens + attn::kAppendRow - 1) / attn::kAppendRow));
    if (dtype == 1) hipLaunchKernelGGL(attn::kv_append_kernel<__bf16>, grid, dim3(kThreads), 0, stream, p);
    else hipLaunchKernelGGL(attn::kv_append_kernel<float>, grid, dim3(kThreads), 0, stream, p);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace ssd
