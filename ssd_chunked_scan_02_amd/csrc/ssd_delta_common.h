// Device helpers shared by the kernels of the gated delta rule: 16x16 MFMA tiles of either element type, operands split
// into bf16 terms, and the chunks of the packed axis.  gfx950 only.
//
// Precision.  bf16 inputs are exact operands of the matrix unit.  What is computed (states, decayed scores, the
// triangular inverse) is fp32, and a bf16 operand is made of it in three terms, each the rounded rest of those before it,
// which together hold an fp32's 24 bits; the product of two such operands takes the six MFMAs whose terms' places add up
// to two at most.  So the states and the fp32 gradients of bf16 inputs are as good as those of fp32 inputs, which go
// through fp32 MFMAs (at a sixteenth of the bf16 rate).  Where only a bf16 output (y, dq, dk) is made of a product, its operands have
// two terms, 2^-16 of each, which leaves that output its own rounding.
#pragma once

#include "ssd_common.h"
#include "ssd_delta_launch.h"

namespace ssd {
namespace delta {

typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kC = kDeltaChunk;

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

// Terms of the operands (S, P and U) that only y is made of: two make its error that of its own rounding to bf16; dy . y, which
// the backward pass takes of it, wants all.
template <typename T> constexpr int terms_of_y(bool backward) { return backward || Mat<T>::kTerms == 1 ? Mat<T>::kTerms : 2; }

template <typename T> __device__ __forceinline__ typename Mat<T>::Frag frag(const T* p) {
    return __builtin_bit_cast(typename Mat<T>::Frag, ld16(p));
}

// Memory from a uniform address on, for loads at a lane's offset (a register for all chunks) and a constant one, so that
// a chunk's loads cost no address arithmetic.  Loads from `bytes` on give zeros and stores there do nothing, without a branch
// (branches between loads would have the compiler wait for all of them).
struct Block {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    __amdgpu_buffer_rsrc_t r;
    __device__ __forceinline__ explicit Block(const void* base, uint32_t bytes = 0xffffffffu)
        : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000)) {}
    // (a constant past the instruction's own field goes through a scalar register)
    __device__ __forceinline__ uint4 load16(uint32_t lane, uint32_t at) const {
        return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)(lane + at % 4096u), (int)(at - at % 4096u), 0));
    }
    template <typename T> __device__ __forceinline__ typename Mat<T>::Frag frag(uint32_t lane, uint32_t at) const {
        return __builtin_bit_cast(typename Mat<T>::Frag, load16(lane, at));
    }
    __device__ __forceinline__ float loadf(uint32_t lane, uint32_t at) const {
        return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, (int)(lane + at % 4096u), (int)(at - at % 4096u), 0));
    }
    // W elements beside each other (1 or 2)
    template <int W, typename T> __device__ __forceinline__ void load(uint32_t lane, T (&x)[W]) const {
        typedef T pair __attribute__((ext_vector_type(2)));
        if constexpr (W * sizeof(T) == 8) {
            const pair v = __builtin_bit_cast(pair, __builtin_amdgcn_raw_buffer_load_b64(r, (int)lane, 0, 0));
            x[0] = v[0];
            x[1] = v[1];
        } else if constexpr (W == 2) {
            const pair v = __builtin_bit_cast(pair, __builtin_amdgcn_raw_buffer_load_b32(r, (int)lane, 0, 0));
            x[0] = v[0];
            x[1] = v[1];
        } else if constexpr (sizeof(T) == 4) {
            x[0] = __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(r, (int)lane, 0, 0));
        } else {
            x[0] = __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(r, (int)lane, 0, 0));
        }
    }
    template <int W, typename T> __device__ __forceinline__ void store(uint32_t lane, const float (&x)[W]) const {
        typedef T pair __attribute__((ext_vector_type(2)));
        if constexpr (W * sizeof(T) == 8)
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, pair{(T)x[0], (T)x[1]}), r, (int)lane, 0, 0);
        else if constexpr (W == 2) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, pair{(T)x[0], (T)x[1]}), r, (int)lane, 0, 0);
        else if constexpr (sizeof(T) == 4) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, (T)x[0]), r, (int)lane, 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, (T)x[0]), r, (int)lane, 0, 0);
    }
};

// A tensor's rows from one chunk of a sequence to the next (or back): rows `pitch` bytes apart, of which `width` are in use.
// Rows past the sequence's end are past its block's.
struct Chunks {
    const char* base;  // of the present chunk
    int64_t step;      // bytes from one chunk to the next
    uint32_t whole, last;
    template <typename T>
    __device__ __forceinline__ Chunks(const T* first, int64_t len, int64_t stride, int width) : base(reinterpret_cast<const char*>(first)) {
        const uint32_t pitch = (uint32_t)(stride * sizeof(T)), used = (uint32_t)(width * sizeof(T));
        step = (int64_t)kC * pitch;
        whole = (uint32_t)(kC - 1) * pitch + used;
        last = len > 0 ? (uint32_t)((len - 1) % kC) * pitch + used : 0;
    }
    __device__ __forceinline__ Block block(bool is_last) const { return Block(base, is_last ? last : whole); }
};

// Two values rounded to bf16, and what is left of them.
__device__ __forceinline__ uint32_t take2(float& a, float& b) {
    typedef __bf16 pair __attribute__((ext_vector_type(2)));
    const uint32_t t = __builtin_bit_cast(uint32_t, pair{(__bf16)a, (__bf16)b});
    a -= __builtin_bit_cast(float, t << 16);
    b -= __builtin_bit_cast(float, t & 0xffff0000u);
    return t;
}

// Four values as TERMS terms, `apart` elements from one term to the next.
template <int TERMS> __device__ __forceinline__ void put4(__bf16* p, int apart, f32x4 x) {
    float a = x[0], b = x[1], c = x[2], d = x[3];
#pragma unroll
    for (int u = 0; u < TERMS; ++u) {
        const uint32_t lo = take2(a, b), hi = take2(c, d);
        st8(p + u * apart, uint2{lo, hi});
    }
}
template <int TERMS> __device__ __forceinline__ void put4(float* p, int, f32x4 x) { *reinterpret_cast<f32x4*>(p) = x; }

// One fragment's values as TERMS fragments, `apart` elements from one term to the next.
template <int TERMS> __device__ __forceinline__ void put_frag(__bf16* p, int64_t apart, float (&x)[8]) {
#pragma unroll
    for (int u = 0; u < TERMS; ++u) {
        uint4 t;
        t.x = take2(x[0], x[1]);
        t.y = take2(x[2], x[3]);
        t.z = take2(x[4], x[5]);
        t.w = take2(x[6], x[7]);
        st16(p + u * apart, t);
    }
}
template <int TERMS> __device__ __forceinline__ void put_frag(float* p, int64_t, float (&x)[4]) {
    st16(p, __builtin_bit_cast(uint4, f32x4{x[0], x[1], x[2], x[3]}));
}

// Operands of CT column tiles from LDS: TB terms of step t, tiles `tile` elements and terms `apart` elements from one to the next.
template <typename T, int CT, int TB> struct Operands {
    using M = Mat<T>;
    typename M::Frag f[CT][TB];
    __device__ __forceinline__ void read(const T* at, int t, int tile, int apart) {
#pragma unroll
        for (int i = 0; i < CT; ++i)
#pragma unroll
            for (int u = 0; u < TB; ++u) f[i][u] = frag(at + i * tile + u * apart + t * M::kK);
    }
    // c[i] + a f[i], a in TA terms: the products of terms whose places add up to less than the larger number of terms.  The
    // tiles' sums are independent, so that they follow each other without a wait.
    template <int TA> __device__ __forceinline__ void add(f32x4 (&c)[CT], const typename M::Frag* a) const {
        constexpr int TOP = TA > TB ? TA : TB;
#pragma unroll
        for (int j = TB - 1; j >= 0; --j)
#pragma unroll
            for (int k = TA - 1; k >= 0; --k)
                if (j + k < TOP)
#pragma unroll
                    for (int i = 0; i < CT; ++i) c[i] = M::mma(a[k], f[i][j], c[i]);
    }
};

// Operand of a chunk's columns from its rows [token][n] in LDS: index n0 + m, contracting over the tokens of step ks.
template <typename T> __device__ __forceinline__ typename Mat<T>::Frag columns_of(const T* rows, int row, int n0, int ks, int m, int g) {
    if constexpr (sizeof(T) == 2) {
        typedef short v4i16 __attribute__((ext_vector_type(4)));
        typedef short v8i16 __attribute__((ext_vector_type(8)));
        typedef __attribute__((address_space(3))) v4i16 lds_v4i16;
        // ds_read_b64_tr_b16: a 16-lane group whose lane 4 r + q points at row r, columns 4 q .. 4 q + 3 returns column i
        // of those four rows in its lane i
        const T* at = rows + (32 * ks + 4 * g + m / 4) * row + n0 + 4 * (m % 4);
        const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)at), hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(at + 16 * row));
        return __builtin_bit_cast(bf16x8, v8i16{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
    } else {
        const T* at = rows + (16 * ks + 4 * g) * row + n0 + m;
        return f32x4{at[0], at[row], at[2 * row], at[3 * row]};
    }
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
// The sequence whose slots hold `slot`, or the last one before it: the last one that begins at most there, found 64
// sequences at a time (one load's wait for 64 sequences, two for 4096).  Called by whole waves.
__device__ __forceinline__ int64_t seq_of_slot(const DeltaParams& p, int64_t slot) {
    const int lane = threadIdx.x % kWave;
    int64_t lo = 0, n = p.nseq;
    while (n > 1) {
        const int64_t step = (n - 1) / kWave + 1, s = lo + step * lane;
        const bool at_most = s < lo + n && span_of(p, s).lo / kC + s <= slot;
        const int cnt = __popcll(__ballot(at_most));
        const int64_t at = cnt > 0 ? step * (cnt - 1) : 0;
        lo += at;
        n = n - at < step ? n - at : step;
    }
    return (int64_t)__builtin_amdgcn_readfirstlane((int)lo);
}

}  // namespace delta
}  // namespace ssd
