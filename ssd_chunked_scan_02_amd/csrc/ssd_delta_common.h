// Device helpers shared by the kernels of the gated delta rule: 16x16 MFMA tiles of either element type, operands split
// into two bf16 terms, and the chunks of the packed axis.  gfx950 only.
//
// Precision.  bf16 inputs are exact operands of the matrix unit.  What is computed (states, decayed scores, the
// triangular inverse) is fp32, and a bf16 operand is made of it in three terms, each the rounded rest of those before it,
// which together hold an fp32's 24 bits; the product of two such operands takes the six MFMAs whose terms' places add up
// to two at most.  So the states and the fp32 gradients of bf16 inputs are as good as those of fp32 inputs, which go
// through fp32 MFMAs (at a sixteenth of the bf16 rate).  Where only a bf16 output is made of a product, its operands have
// one term or two.
#pragma once

#include "ssd_common.h"
#include "ssd_delta_launch.h"

namespace ssd {
namespace delta {

typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kC = kDeltaChunk;
constexpr int kCols = kDeltaCols;

// An operand fragment is 16 bytes a lane: lane 16 g + m holds row (column) m, contraction indices kE g .. of kK.  The
// accumulator of a 16x16 tile has row 4 g + r, column m in register r.  Contractions over a chunk's tokens take them in
// the order in which two (bf16) stacked accumulators hold them, so that these are operands as they are: index kE g + e
// of step ks is token token_of(ks, g, e), and an accumulator's four rows go to place_of(tile, g) and the three after it.
template <typename T> struct Mat;
template <> struct Mat<__bf16> {
    using Frag = bf16x8;
    static constexpr int kE = 8, kK = 32, kTerms = 3, kPad = 8;
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) { return mfma_bf16(a, b, c); }
    static __device__ __forceinline__ int token_of(int ks, int g, int e) { return 32 * ks + 16 * (e / 4) + 4 * g + e % 4; }
    static __device__ __forceinline__ int place_of(int tile, int g) { return 32 * (tile / 2) + 8 * g + 4 * (tile % 2); }
};
template <> struct Mat<float> {
    using Frag = f32x4;
    static constexpr int kE = 4, kK = 16, kTerms = 1, kPad = 4;
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c = mfma_f32(a[i], b[i], c);
        return c;
    }
    static __device__ __forceinline__ int token_of(int ks, int g, int e) { return 16 * ks + 4 * g + e; }
    static __device__ __forceinline__ int place_of(int tile, int g) { return 16 * tile + 4 * g; }
};

template <typename T> __device__ __forceinline__ typename Mat<T>::Frag frag(const T* p) {
    return __builtin_bit_cast(typename Mat<T>::Frag, ld16(p));
}

// Rows of a tensor from `base` on, `stride` elements apart, `width` elements of each in use: loads from row `have` on give
// zeros and stores there do nothing, without a branch (branches between loads would have the compiler wait for all of them).
template <typename T> struct Rows {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    __amdgpu_buffer_rsrc_t r;
    uint32_t pitch;
    __device__ __forceinline__ Rows(const T* base, int64_t have, int64_t stride, int width) {
        pitch = (uint32_t)(stride * sizeof(T));
        r = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(base), (short)0,
                                              have > 0 ? (int)((uint32_t)(have - 1) * pitch + (uint32_t)(width * sizeof(T))) : 0, 0x00020000);
    }
    __device__ __forceinline__ int at(int row, int col) const { return (int)((uint32_t)row * pitch + (uint32_t)(col * sizeof(T))); }
    __device__ __forceinline__ typename Mat<T>::Frag frag(int row, int col) const {
        return __builtin_bit_cast(typename Mat<T>::Frag, __builtin_amdgcn_raw_buffer_load_b128(r, at(row, col), 0, 0));
    }
    // two elements beside each other
    __device__ __forceinline__ void load2(int row, int col, T (&x)[2]) const {
        if constexpr (sizeof(T) == 2) {
            typedef T pair __attribute__((ext_vector_type(2)));
            const pair v = __builtin_bit_cast(pair, __builtin_amdgcn_raw_buffer_load_b32(r, at(row, col), 0, 0));
            x[0] = v[0];
            x[1] = v[1];
        } else {
            const f32x2 v = __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(r, at(row, col), 0, 0));
            x[0] = v[0];
            x[1] = v[1];
        }
    }
    __device__ __forceinline__ void store2(int row, int col, float a, float b) const {
        if constexpr (sizeof(T) == 2) {
            typedef T pair __attribute__((ext_vector_type(2)));
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, pair{(T)a, (T)b}), r, at(row, col), 0, 0);
        } else {
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, f32x2{a, b}), r, at(row, col), 0, 0);
        }
    }
};

// Four values as TERMS terms, `apart` elements from one term to the next.
template <int TERMS> __device__ __forceinline__ void put4(__bf16* p, int apart, f32x4 x) {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int u = 0; u < TERMS; ++u) {
        bf16x4 t;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t[i] = (__bf16)x[i];
            x[i] -= (float)t[i];
        }
        *reinterpret_cast<bf16x4*>(p + u * apart) = t;
    }
}
template <int TERMS> __device__ __forceinline__ void put4(float* p, int, f32x4 x) { *reinterpret_cast<f32x4*>(p) = x; }

// One fragment's values as TERMS fragments, `apart` elements from one term to the next.
template <int TERMS> __device__ __forceinline__ void put_frag(__bf16* p, int64_t apart, float (&x)[8]) {
#pragma unroll
    for (int u = 0; u < TERMS; ++u) {
        bf16x8 t;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            t[i] = (__bf16)x[i];
            x[i] -= (float)t[i];
        }
        st16(p + u * apart, __builtin_bit_cast(uint4, t));
    }
}
template <int TERMS> __device__ __forceinline__ void put_frag(float* p, int64_t, float (&x)[4]) {
    st16(p, __builtin_bit_cast(uint4, f32x4{x[0], x[1], x[2], x[3]}));
}

// c + a b with a in TA terms and b in TB, in memory `apart` elements apart: the products of terms whose places add up to
// less than the larger number of terms.
template <typename T, int TA, int TB>
__device__ __forceinline__ f32x4 mma_terms(const typename Mat<T>::Frag* a, const T* b, int apart, f32x4 c) {
    constexpr int TOP = TA > TB ? TA : TB;
#pragma unroll
    for (int j = TB - 1; j >= 0; --j) {
        const typename Mat<T>::Frag x = frag(b + j * apart);
#pragma unroll
        for (int i = TA - 1; i >= 0; --i)
            if (i + j < TOP) c = Mat<T>::mma(a[i], x, c);
    }
    return c;
}

// Sum over the 16 lanes that share a lane group g (one row of an accumulator).
__device__ __forceinline__ float sum16(float x) {
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) x += __shfl_xor(x, off, kWave);
    return x;
}

struct Span {
    int64_t lo, len;
};
// Tokens of sequence s, its offsets clamped into the axis.
__device__ __forceinline__ Span span_of(const DeltaParams& p, int64_t s) {
    if (!p.cu) return Span{s * p.each, p.each};
    int64_t lo = p.cu[s], hi = p.cu[s + 1];
    lo = lo < 0 ? 0 : lo > p.total ? p.total : lo;
    hi = hi < lo ? lo : hi > p.total ? p.total : hi;
    return Span{lo, hi - lo};
}
// The sequence whose slots hold `slot`, or the last one before it.
__device__ __forceinline__ int64_t seq_of_slot(const DeltaParams& p, int64_t slot) {
    int64_t a = 0, b = p.nseq - 1;
    while (a < b) {
        const int64_t m = (a + b + 1) / 2;
        if (span_of(p, m).lo / kC + m <= slot) a = m;
        else b = m - 1;
    }
    return a;
}

}  // namespace delta
}  // namespace ssd
