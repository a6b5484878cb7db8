// Device helpers shared by the attention kernels: 32x32 MFMA tiles of either element type, the LDS
// tile layout they read, sequence lookup on the packed axes, and the bucket table.  gfx950 only.
//
// Every product here is arranged so that one operand's second index (a query in the forward and
// query-gradient kernels, a key in the key-gradient kernel) is the MFMA column, lane % 32: the
// softmax statistics of that index are then one number per lane, and the accumulator registers of
// a score tile are, without any exchange between lanes, the operand of the next product that
// contracts over its rows.  Accumulator register r of lane half h holds row (r % 4) + 8 (r / 4) +
// 4 h; the LDS reads of the other operand take their rows in the same order.
#pragma once

#include "ssd_attn_launch.h"
#include "ssd_common.h"

namespace ssd {
namespace attn {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef short v8i16 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// start of a running maximum (log2 units): below any finite score, and finite, so that a row that
// has seen nothing but masked scores (minus infinity) takes exp2(-inf) = 0 and not a NaN
constexpr float kNoMax = -1e30f;
// Rows of the query axis.  The heads of a group meet the same keys, so that a tile may hold all of them:
// row R is query R / pack, head R % pack of the group (pack 1: a tile is of one head).  Keys and values
// are then read once for the group, and tiles are of fewer queries, which wastes less on short documents
// and on the diagonal.
//
// Rows of a workgroup's own tile.  With enough work for the chip each of its four waves owns 32 rows and they
// share what they stream.  With too little (SPLIT) all four own the same 32 rows, each streams every
// fourth tile through LDS of its own, and their results are joined at the end: four times the
// workgroups, and a quarter of the way for each.
template <bool SPLIT> constexpr int kOwn = SPLIT ? 32 : 128;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// One operand fragment is 16 bytes a lane: kK contraction steps over both lane halves.
template <typename T> struct Op;
template <> struct Op<__bf16> {
    using Frag = bf16x8;
    static constexpr int kE = 8, kK = 16, kKT = 64;  // kKT: rows of a streamed LDS tile
    static __device__ __forceinline__ f32x16 mma(Frag a, Frag b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    // accumulator rows kK * kk ... of a 32-row tile as an operand, rounded once to bf16: the
    // matrix unit's operand type (products and sums stay fp32)
    static __device__ __forceinline__ Frag pack(const f32x16& v, int kk) {
        Frag f;
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = (__bf16)v[8 * kk + j];
        return f;
    }
};
template <> struct Op<float> {
    using Frag = f32x4;
    static constexpr int kE = 4, kK = 8, kKT = 32;
    static __device__ __forceinline__ f32x16 mma(Frag a, Frag b, f32x16 c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ Frag pack(const f32x16& v, int kk) {
        return Frag{v[4 * kk], v[4 * kk + 1], v[4 * kk + 2], v[4 * kk + 3]};
    }
};

// c plus the sum of a bf16 operand's eight elements, in fp32.
__device__ __forceinline__ float sum_of(bf16x8 f, float c) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 one = {(__bf16)1.f, (__bf16)1.f};
#pragma unroll
    for (int i = 0; i < 8; i += 2) c = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{f[i], f[i + 1]}, one, c, false);
    return c;
}

// Row-major tile [rows][D] in LDS, in 16-byte chunks, chunk c of a row stored at c ^ swz(row).  LDS serves
// 256 bytes (16 chunks) at a time: the 16 rows that a pass of 16-byte reads takes at one chunk, and the
// four rows by four chunks that a pass of transposing reads takes, lie in different banks without padding.
// (fp32: a pass of 4-byte reads takes eight chunks of two rows four apart.)  swz only moves bits of the
// row, so that swz(a ^ b) = swz(a) ^ swz(b).
template <typename T, int D> struct Tile {
    static constexpr int kE = Op<T>::kE;
    static constexpr int CH = D / kE;
    static constexpr int RB = D * (int)sizeof(T);
    static __host__ __device__ __forceinline__ constexpr int swz(int r) {
        if constexpr (sizeof(T) == 2)
            return CH == 16 ? ((r & 3) << 2) | ((r >> 2) & 3) : CH == 8 ? ((r & 2) << 1) | ((r >> 2) & 3) : (r >> 2) & 3;
        else
            return CH >= 16 ? ((r & 4) << 1) | ((r & 3) << 1) | ((r >> 3) & 1) : (r >> 1) & 7;
    }
    static __device__ __forceinline__ int at(int row, int c) { return (row * CH + (c ^ swz(row))) * kE; }

    // A lane's part of the byte addresses of its operands: rows() and cols() add to it what does not depend on
    // the lane, by one xor (the swizzle's bits and a chunk's are the same ones) and an immediate offset.
    struct Lanes {
        uint32_t row, col;
        __device__ __forceinline__ explicit Lanes(int lane) {
            const int r = lane % 32, h = lane / 32;
            row = (uint32_t)(r * RB + (h ^ swz(r)) * 16);
            if constexpr (sizeof(T) == 2) {
                const int q = lane % 4, kr = 4 * h + (lane % 16) / 4;
                col = (uint32_t)(kr * RB + ((2 * ((lane / 16) % 2) + q / 2) ^ swz(kr)) * 16 + (q % 2) * 8);
            } else {
                col = (uint32_t)(4 * h * RB + (((lane % 32) * 4) ^ (swz(4 * h) * 16)));
            }
        }
        // Keeps the compiler from holding every address of a loop in a register of its own.
        __device__ __forceinline__ void renew() { asm volatile("" : "+v"(row), "+v"(col)); }
    };

    // operand whose index is a row (lane % 32 of row0 .., a multiple of 32), contracting over columns kK * t ..
    static __device__ __forceinline__ typename Op<T>::Frag rows(const T* s, int row0, int t, const Lanes& z) {
        return __builtin_bit_cast(typename Op<T>::Frag, ld16(reinterpret_cast<const char*>(s) + (z.row ^ (32u * t)) + row0 * RB));
    }
    // operand whose index is a column (lane % 32 of col0 .., a multiple of 32), contracting over rows
    // row0 + kK * kk .. in the row order of an accumulator (see the top of this file)
    static __device__ __forceinline__ typename Op<T>::Frag cols(const T* s, int row0, int kk, int col0, const Lanes& z) {
        const char* at = reinterpret_cast<const char*>(s);
        if constexpr (sizeof(T) == 2) {
            // ds_read_b64_tr_b16: a 16-lane group whose lane 4 r + q points at row r, columns 4 q .. 4 q + 3
            // returns column i of those four rows in its lane i
            const uint32_t low = z.col ^ (uint32_t)(2 * col0);
            at += (row0 + 16 * kk) * RB;
            const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(at + low));
            const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(at + (low ^ (swz(8) * 16u)) + 8 * RB));
            const v8i16 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            return __builtin_bit_cast(bf16x8, v);
        } else {
            f32x4 v;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = *reinterpret_cast<const float*>(at + (z.col ^ (uint32_t)(swz(8 * kk + i) * 16) ^ (uint32_t)(4 * col0)) +
                                                       (row0 + 8 * kk + i) * RB);
            return v;
        }
    }
};

// What the kernels know a wave's outstanding memory operations by (s_waitcnt of gfx9: vmcnt in bits 3:0 and
// 15:14, expcnt in 6:4, lgkmcnt in 11:8): everything loaded to LDS has arrived, and with kAll every LDS
// read has returned too.
constexpr int kLoadsDone = 0x0F70, kAllDone = 0x0070;

// Streams ROWS-row tiles of a [tokens][stride] tensor into LDS by THREADS threads, with loads that write LDS
// themselves (global_load_lds_dwordx4): 16 bytes a lane land in lane order behind a wave's LDS address, so
// the chunk order of Tile is made on the global side.  A thread's byte offsets within a tile do not
// change, so a whole tile costs no address arithmetic; in a last, partial tile the rows past the end are
// read as the last row (a copy of a real row, whose weight is zero).
template <typename T, int D, int ROWS, int THREADS> struct Feed {
    using L = Tile<T, D>;
    static constexpr int kLoads = ROWS * L::CH / THREADS;
    static_assert(ROWS * L::CH % THREADS == 0, "every thread loads whole chunks");
    typedef const __attribute__((address_space(1))) void* Global;
    typedef __attribute__((address_space(3))) void* Local;
    uint32_t off[kLoads];
    uint32_t pitch;  // bytes from one token to the next

    static __device__ __forceinline__ int row(int i) { return ((int)threadIdx.x % THREADS + THREADS * i) / L::CH; }
    static __device__ __forceinline__ uint32_t col(int i) {
        const int c = ((int)threadIdx.x % THREADS + THREADS * i) % L::CH;
        return (uint32_t)(c ^ L::swz(row(i))) * 16u;
    }
    __device__ __forceinline__ void init(int64_t stride) {
        pitch = (uint32_t)(stride * (int64_t)sizeof(T));
#pragma unroll
        for (int i = 0; i < kLoads; ++i) off[i] = (uint32_t)row(i) * pitch + col(i);
    }
    // Takes the infinities and NaN out of what this thread has loaded, rows `at` .. of the sequence, and notes for their
    // columns the first row with a NaN, an infinity and a negative infinity.
    static __device__ __forceinline__ void clean(T* s, int at, int (*first)[D]) {
        const int wave = (int)threadIdx.x % THREADS / kWave, lane = threadIdx.x % kWave;
#pragma unroll 1
        for (int i = 0; i < kLoads; ++i) {
            T* chunk = s + (wave * kWave + THREADS * i + lane) * L::kE;
#pragma unroll 1
            for (int e = 0; e < L::kE; ++e) {
                const float x = (float)chunk[e];
                if (fabsf(x) < INFINITY) continue;
                chunk[e] = (T)0.f;
                atomicMin(&first[x != x ? 0 : x > 0.f ? 1 : 2][col(i) / (int)sizeof(T) + e], at + row(i));
            }
        }
    }
    // rows 0 .. of `g`, the tensor's row `first`; `left` >= 1 rows are there
    __device__ __forceinline__ void load(T* s, const T* g, int first, int left) const {
        const char* base = reinterpret_cast<const char*>(g) + (int64_t)first * pitch;
        const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x % THREADS / kWave);
        if (left >= ROWS) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                __builtin_amdgcn_global_load_lds((Global)(base + off[i]), (Local)(s + (wave * kWave + THREADS * i) * L::kE), 16, 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                __builtin_amdgcn_global_load_lds((Global)(base + (uint32_t)min(row(i), left - 1) * pitch + col(i)),
                                                 (Local)(s + (wave * kWave + THREADS * i) * L::kE), 16, 0, 0);
        }
    }
};

// Row of accumulator register r in the lower lane half (the upper half: + 4).
__device__ __forceinline__ constexpr int acc_row(int r) { return (r % 4) + 8 * (r / 4); }

// The other lane half's value.
__device__ __forceinline__ float other_half(float v) { return __shfl_xor(v, 32, kWave); }

// A sequence of the packed axes and one tile of its queries or keys.
struct Span {
    int64_t q0, k0;  // first query and key row
    int lq, lk;      // their numbers
    int rows;        // query rows: lq * pack
    int tile;        // tile of the axis the slots count; negative: the slot is empty
    int seq;
    int slot;        // place of the tile in the axis's own order
};

__device__ __forceinline__ int64_t clamp64(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : (v > hi ? hi : v); }

// Offset s as a call gave it, clamped into the axis, so that no offsets lead outside a tensor.
__device__ __forceinline__ int offset_at(const int64_t* cu, int64_t s, int total) { return (int)clamp64(cu[s], 0, total); }

// The last s in [0, nseq) with start(s) <= x, 64 sequences at a time: one step for 64 sequences, two for
// 4096.  Called by whole waves.
template <typename F> __device__ __forceinline__ int last_at_most(int nseq, F le) {
    const int lane = threadIdx.x % kWave;
    int lo = 0, n = nseq;
    while (n > 1) {
        const int step = (n - 1) / kWave + 1;
        const int64_t s = lo + (int64_t)step * lane;
        const int cnt = __popcll(__ballot(s < lo + n && le((int)s)));
        const int at = cnt > 0 ? step * (cnt - 1) : 0;
        lo += at;
        n = min(n - at, step);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// Sequence and tile of a slot.  Sequence s owns the slots from floor(cu[s] / own) + s on, one more than
// its whole tiles at most, so that a workgroup finds its work from the offsets alone, with no list made
// on the way; a list (p.plan_q, p.plan_k) orders the slots by their work instead.
// (own: rows of a tile; by_keys: the slots count tiles of the key axis)
__device__ __forceinline__ Span find_span(const AttnParams& p, int slot, int own, bool by_keys) {
    const int64_t* cu = by_keys ? p.cu_k : p.cu_q;
    const int2* plan = by_keys ? p.plan_k : p.plan_q;
    const int tq = (int)p.total_q, tk = (int)p.total_k, pack = by_keys ? 1 : p.pack;
    Span sp{};
    int s, tile;
    sp.slot = slot;
    if (plan) {
        const int2 e = plan[slot];
        s = __builtin_amdgcn_readfirstlane(e.x);
        tile = __builtin_amdgcn_readfirstlane(e.y);
        if (tile < 0) {  // (an empty slot's entry is its place and not a sequence)
            sp.slot = s;
            sp.tile = -1;
            return sp;
        }
        sp.slot = (int)((int64_t)offset_at(cu, s, by_keys ? tk : tq) * pack / own) + s + tile;
    } else if (!cu) {
        const int per = by_keys ? p.each_k_tiles : p.each_q_tiles;
        s = (int)((uint32_t)slot / (uint32_t)per);
        tile = slot - s * per;
    } else {
        const int total = by_keys ? tk : tq;
        auto start = [&](int i) { return (int)((int64_t)offset_at(cu, i, total) * pack / own) + i; };
        s = last_at_most((int)p.nseq, [&](int i) { return start(i) <= slot; });
        tile = slot - start(s);
    }
    sp.seq = s;
    int q0, k0;
    if (p.cu_q) {
        q0 = offset_at(p.cu_q, s, tq);
        sp.lq = max(offset_at(p.cu_q, s + 1, tq) - q0, 0);
    } else {
        sp.lq = p.each_q;
        q0 = s * sp.lq;
    }
    if (p.cu_k) {
        k0 = offset_at(p.cu_k, s, tk);
        sp.lk = max(offset_at(p.cu_k, s + 1, tk) - k0, 0);
    } else {
        sp.lk = p.each_k;
        k0 = s * sp.lk;
    }
    sp.q0 = q0;
    sp.k0 = k0;
    sp.rows = sp.lq * pack;
    const int len = by_keys ? sp.lk : sp.rows;
    sp.tile = tile >= 0 && (int64_t)tile * own < len ? tile : -1;
    return sp;
}

// Heads in a query tile: a group's, except with a bucket table, whose bias in LDS and sums by distance are
// of one head (and rows are counted in 32 bits).
inline int query_pack(const AttnParams& p, int bias) {
    const int group = p.H / p.Hk;
    return bias == kBiasBuckets || p.total_q * group >= ((int64_t)1 << 31) - 1024 ? 1 : group;
}
inline int64_t query_slots(const AttnParams& p, int own) {
    // (equal sequences: their rows have to be counted one by one)
    return attn_slots(p.cu_q, p.total_q * p.pack, p.nseq, own);
}
// Lengths and tiles of equal sequences.
inline void set_each(AttnParams& p, int q_own, int k_own) {
    p.each_q = p.nseq ? (int)(p.total_q / p.nseq) : 0;
    p.each_k = p.nseq ? (int)(p.total_k / p.nseq) : 0;
    p.each_q_tiles = (int)(((int64_t)p.each_q * p.pack + q_own - 1) / q_own);
    p.each_k_tiles = (p.each_k + k_own - 1) / k_own;
}

// Workgroup -> (slot, head).  Heads run fastest, the slots from the last (under a causal mask the
// longest) to the first.  Workgroups reach the 8 XCDs in turn, so with 8 or more heads an XCD keeps a
// run of neighbouring heads, which share keys and values in its L2.
__device__ __forceinline__ void work_item(uint32_t id, int slots, uint32_t H, int& slot, int& head) {
    const uint32_t at = id / H, x = id - at * H;
    slot = slots - 1 - (int)at;
    head = (int)(H % 8 == 0 ? (x % 8) * (H / 8) + x / 8 : x);
}

// Two neighbouring groups of four accumulator rows (r .. r + 3 and r + 4 .. r + 7) of a 32-row tile hold, over
// both lane halves, rows 2 r .. 2 r + 7 and 2 r + 8 .. 2 r + 15.  Swapping one against the other between the halves
// gives each lane eight rows in a row: 2 r + 8 half .., one 16-byte store in bf16 (two in fp32).
template <typename T> __device__ __forceinline__ void store_rows(T* out, const f32x16& v, int r, int half, float f) {
    if constexpr (sizeof(T) == 2) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)(v[r + 2 * i] * f), (__bf16)(v[r + 2 * i + 1] * f)});
        // (word i of the first group against word i of the second: the first's upper lanes for the second's lower)
        const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
        const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
        st16(out + 2 * r + 8 * half, uint4{a[0], b[0], a[1], b[1]});
    } else {
        store4(out + 2 * r + 4 * half, v[r] * f, v[r + 1] * f, v[r + 2] * f, v[r + 3] * f);
        store4(out + 2 * r + 8 + 4 * half, v[r + 4] * f, v[r + 5] * f, v[r + 6] * f, v[r + 7] * f);
    }
}

// Bucket of a relative position (key - query) of at most max_distance.
__device__ __forceinline__ int bucket_of(const AttnBuckets& b, int rel) {
    if (b.both) return b.of[abs(rel)] + (rel > 0 ? b.nborders + 1 : 0);
    return b.of[rel < 0 ? -rel : 0];
}

// The head's bias, in log2 units, of relative positions -max_distance .. max_distance.
__device__ __forceinline__ void fill_bias(float* lut, const AttnParams& p, int head) {
    const int m = p.bk.max_distance;
    for (int i = threadIdx.x; i <= 2 * m; i += kThreads) lut[i] = p.table[(int64_t)bucket_of(p.bk, i - m) * p.H + head] * kLog2e;
}

// What turns a raw product x = q.k into a score in log2 units, and the derivative of the cap.
//   no cap: x * a, a = scale log2 e
//   cap c:  c tanh(x scale / c) log2 e
struct Score {
    float a;       // no cap: scale log2 e; cap: 2 scale log2 e / c (bf16) or scale / c (fp32)
    float c2;      // c log2 e
    float rc2;     // 1 / c2
    float k[4];    // cap, bf16: c2 tanh(x scale / c) = x (k0 + k1 x^2 + k2 x^4 + k3 x^6) where x^2 <= small
    float small;
    float none;    // a masked score; raw (no bias): a masked product, or with a cap a score whose derivative is finite
    template <typename T> __device__ __forceinline__ void init(float scale, float cap, bool capped, bool raw = false) {
        // (a scale of zero: a finite factor times a masked score has to stay minus infinity)
        const float s = fabsf(scale) < 1e-30f ? 1e-30f : scale, u = capped ? s / cap : 0.f;
        c2 = cap * kLog2e;
        rc2 = capped ? 1.f / c2 : 0.f;
        // (finite, so that a product of zero is a score of zero)
        a = !capped ? s * kLog2e : fminf(fmaxf(sizeof(T) == 4 ? u : 2.f * u * kLog2e, -3e38f), 3e38f);
        k[0] = s * kLog2e;
        k[1] = k[0] * u * u * (-1.f / 3.f);
        k[2] = k[0] * (u * u) * (u * u) * (2.f / 15.f);
        k[3] = k[0] * (u * u) * (u * u) * (u * u) * (-17.f / 315.f);
        // (capped: lse is at least -c2, so that its weight, under 2^-160, is zero; and (160 / c2)^2 is finite from caps
        // of 2^-56 on)
        none = raw && capped ? -2.f * c2 - 160.f : raw && s < 0.f ? INFINITY : -INFINITY;
        // (a cap so far below the scale that the series' factors overflow: the other form, off by 1e-7 of that cap)
        small = capped && fabsf(k[3]) < 1e38f ? 0.0625f / (u * u) : -1.f;
    }
    // tanh by its series, for arguments within 1/4 (the next term, 62/2835 u^9, is under 4e-7 of u there): 5 full-rate
    // operations.
    __device__ __forceinline__ float series(float x) const {
#pragma clang fp contract(off)
        const float q = x * x;
        return x * __builtin_fmaf(q, __builtin_fmaf(q, __builtin_fmaf(q, k[3], k[2]), k[1]), k[0]);
    }
    // tanh u = 1 - 2 / (1 + e^2u) from the hardware's exp2 and reciprocal, which the unit for them takes 8 times as long
    // for.  It is off by some 1e-7 of the cap, whatever u: for arguments past 1/4 only.
    __device__ __forceinline__ float saturating(float x) const {
#pragma clang fp contract(off)
        return __builtin_fmaf(-2.f * c2, __builtin_amdgcn_rcpf(1.f + exp2_hw(x * a)), c2);
    }
    // The capped scores of N vectors of products, in place.  bf16: each by the form for its own argument, so that a score
    // does not depend on the others; a wave whose arguments are all small leaves the other form out.  fp32: the math
    // library's tanh.
    template <typename T, typename V, int N> __device__ __forceinline__ void capped(V (&s)[N]) const {
        constexpr int L = sizeof(V) / 4;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int r = 0; r < L; ++r) s[n][r] = c2 * tanhf(s[n][r] * a);
        } else {
            float most = 0.f;
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int r = 0; r < L; ++r) most = fmaxf(most, fabsf(s[n][r]));
            if (__all(most * most <= small)) {
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int r = 0; r < L; ++r) s[n][r] = series(s[n][r]);
            } else {
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int r = 0; r < L; ++r) {
                        float x = s[n][r];
                        x = x * x <= small ? series(x) : saturating(x);
                        asm volatile("" : "+v"(x));  // (one after the other: side by side they cost the tile loop a wave a SIMD)
                        s[n][r] = x;
                    }
            }
        }
    }
    // derivative of the cap at a capped score
    __device__ __forceinline__ float slope(float s) const {
        const float t = s * rc2;
        return 1.f - t * t;
    }
};

// 16 bytes of a query for the forward pass, with the sign of the scale: its maxima are taken of raw products,
// whose factor has to be positive then.
template <typename T> __device__ __forceinline__ typename Op<T>::Frag signed_frag(const T* g, float scale) {
    typename Op<T>::Frag f = __builtin_bit_cast(typename Op<T>::Frag, ld16(g));
    if (scale < 0.f) f = -f;
    return f;
}

// Adds the bias to scores s, N 32-row blocks whose register 0 has relative position rel (key - query), and
// register r STEP * acc_row(r) further on (block n: STEP * 32 n).  Factor a on the scores first.  [lowest, highest]:
// relative positions in any lane.  Returns whether some of them are nearer than the table's reach.
template <int BIAS, int STEP, int N>
__device__ __forceinline__ bool add_bias(f32x16 (&s)[N], float a, float slope2, const float* lut, int md, int rel, int lowest,
                                         int highest) {
    if constexpr (BIAS == kBiasSlopes) {
        const float at = (float)rel;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                s[n][r] = s[n][r] * a - slope2 * fabsf(at + (float)(STEP * (32 * n + acc_row(r))));
        return true;
    } else if constexpr (BIAS == kBiasBuckets) {
        if (highest <= -md || lowest >= md) {
            const float b = lut[highest <= -md ? 0 : 2 * md];
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int r = 0; r < 16; ++r) s[n][r] = s[n][r] * a + b;
            return false;
        }
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                s[n][r] = s[n][r] * a + lut[min(max(rel + STEP * (32 * n + acc_row(r)), -md), md) + md];
        return true;
    } else {
        return true;
    }
}

// Joins the four waves' accumulators of the same 32 rows (SPLIT), each weighted by w[wave][row] where w is given.  A
// wave keeps its own in one of the four regions that two of the kernel's tile arrays give; the sums of row
// `row`, columns d .. d + 3 come out for thread (row, d / 4).
template <typename T, int D> struct Join {
    static constexpr int kRegion = 32 * D;  // floats
    static constexpr int kPer = (int)sizeof(T);  // regions in one array of 4 x 32 x D elements
    static __device__ __forceinline__ float* region(T* a, T* b, int wave) {
        return reinterpret_cast<float*>(wave < kPer ? a : b) + (wave % kPer) * kRegion;
    }
    static __device__ __forceinline__ int place(int row, int d4) { return row * D + 4 * (d4 ^ (row % 8)); }
    static __device__ __forceinline__ void keep(T* a, T* b, const f32x16 (&acc)[D / 32], int lane, int wave) {
        float* mine = region(a, b, wave);
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
            for (int r = 0; r < 16; r += 4)
                *reinterpret_cast<f32x4*>(mine + place(lane % 32, 8 * d + r / 2 + lane / 32)) =
                    f32x4{acc[d][r], acc[d][r + 1], acc[d][r + 2], acc[d][r + 3]};
    }
    static __device__ __forceinline__ f32x4 sum(T* a, T* b, int row, int d4, const float* w) {
        f32x4 v{};
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(region(a, b, i) + place(row, d4));
            v += w ? w[32 * i + row] * x : x;
        }
        return v;
    }
};

}  // namespace attn
}  // namespace ssd
