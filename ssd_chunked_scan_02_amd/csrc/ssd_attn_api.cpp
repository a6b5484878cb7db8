// C ABI of the attention operators (declared in include/ssd_attn.h): argument validation, workspace
// sizing and dispatch to the kernels.  Every check runs before the first HIP call.
#include "ssd_attn.h"

#include <cmath>

#include <hip/hip_runtime.h>

#include "ssd_attn_launch.h"

namespace {

// one token axis: in-sequence positions, and positions one tile past an end, are 32-bit in the kernels
constexpr int64_t kMaxTokens = ((int64_t)1 << 31) - 1025;
constexpr int64_t kMaxHeads = 1 << 16;

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// A whole number (little-endian 32-bit limbs), so that bucket borders are compared without rounding.  The
// largest is 1025^32 * 32^32, under 2^481.
struct Whole {
    uint32_t limb[16] = {1};
    void times_power(uint32_t f, int n) {
        while (n-- > 0) {
            uint64_t carry = 0;
            for (uint32_t& x : limb) {
                carry += (uint64_t)x * f;
                x = (uint32_t)carry;
                carry >>= 32;
            }
        }
    }
    bool at_least(const Whole& o) const {
        for (int i = 15; i >= 0; --i)
            if (limb[i] != o.limb[i]) return limb[i] > o.limb[i];
        return true;
    }
};

// Is bucket e + k reached at distance d, (d / e)^f >= (m / e)^k, that is d^f e^k >= m^k e^f?
bool reached(int d, int e, int f, int m, int k) {
    Whole a, b;
    a.times_power((uint32_t)d, f);
    a.times_power((uint32_t)e, k);
    b.times_power((uint32_t)m, k);
    b.times_power((uint32_t)e, f);
    return a.at_least(b);
}

// The distances at which a direction's bucket goes up by one: e - 1 of them one apart, then f.
int make_buckets(ssd::AttnBuckets& out, int num_buckets, int max_distance, int both) {
    if (both != 0 && both != 1) return SSD_ERR_INVALID;
    const int n = both ? num_buckets / 2 : num_buckets;
    if (num_buckets < (both ? 4 : 2) || (both && num_buckets % 2 != 0) || n > ssd::kMaxBorders) return SSD_ERR_INVALID;
    const int e = n / 2, f = n - e;
    if (max_distance <= e) return SSD_ERR_INVALID;
    if (max_distance > ssd::kMaxDistance) return SSD_ERR_UNSUPPORTED;
    out.total = num_buckets;
    out.both = both;
    out.max_distance = max_distance;
    out.nborders = n - 1;
    int at = 0;
    for (int d = 1; d < e; ++d) out.borders[at++] = d;
    for (int k = 0; k < f; ++k) {
        // the smallest d with d >= e (m / e)^(k / f): from the power where it is clearly between two
        // whole numbers, by the exact comparison where it is next to one
        const double x = e * std::pow((double)max_distance / e, (double)k / f);
        int d = (int)std::ceil(x);
        const int near = (int)std::llround(x);
        if (std::fabs(x - near) < 1e-9 * x) d = reached(near, e, f, max_distance, k) ? near : near + 1;
        out.borders[at++] = d;
    }
    for (int d = 0, b = 0; d <= max_distance; ++d) {
        while (b < out.nborders && out.borders[b] <= d) ++b;
        out.of[d] = (uint8_t)b;
    }
    return SSD_OK;
}

int check_shape(int64_t H, int64_t Hk, int64_t D, int32_t dtype) {
    if (H < 1 || Hk < 1 || H > kMaxHeads || H % Hk != 0 || D < 1) return SSD_ERR_INVALID;
    if (dtype != SSD_F32 && dtype != SSD_BF16) return SSD_ERR_INVALID;
    if (D != 32 && D != 64 && D != 128) return SSD_ERR_UNSUPPORTED;
    if (H * D >= ((int64_t)1 << 24)) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// The cap as the kernels take it, within [2^-56, 2^96], where their 1 / cap^2 and cap log2 e are finite.  Scores under a
// cap of 2^-56 are zero to the last bit of an fp32 weight, and 2^96 caps none that fp32 products of use reach.
float take_cap(float cap) {
    return cap > 0.f ? std::fmin(std::fmax(cap, 0x1p-56f), 0x1p96f) : 0.f;
}

int check_stride(int64_t given, int64_t dense, int64_t elem, int64_t& out) {
    if (given == 0) {
        out = dense;
        return SSD_OK;
    }
    // (a tile's byte offsets are 32-bit: 64 rows of up to 2^24 four-byte elements)
    if (given < dense || given >= ((int64_t)1 << 24)) return SSD_ERR_INVALID;
    if (given * elem % 16 != 0) return SSD_ERR_ALIGN;
    out = given;
    return SSD_OK;
}

// Everything that forward and backward check alike; fills the launch parameters they share.
int fill(const ssd_attn_dims* d, const int64_t* cu_q, const int64_t* cu_k, const int64_t* prefix, const void* q,
         const void* k, const void* v, const float* slopes, const float* table, ssd::AttnParams& p, int& bias) {
    if (!d) return SSD_ERR_INVALID;
    int rc = check_shape(d->nheads, d->nkvheads, d->headdim, d->dtype);
    if (rc != SSD_OK) return rc;
    if (d->nseq < 0 || d->nseq > kMaxTokens || d->total_q < 0 || d->total_q > kMaxTokens || d->total_k < 0 ||
        d->total_k > kMaxTokens)
        return SSD_ERR_INVALID;
    if ((d->causal != 0 && d->causal != 1) || !std::isfinite(d->scale) || !std::isfinite(d->softcap) || d->softcap < 0.f)
        return SSD_ERR_INVALID;
    if (d->nseq > 0 && !cu_q && (d->total_q % d->nseq != 0 || cu_k || d->total_k % d->nseq != 0)) return SSD_ERR_INVALID;
    if (cu_q && !cu_k && d->total_k != d->total_q) return SSD_ERR_INVALID;
    if ((prefix && !d->causal) || (slopes && table)) return SSD_ERR_INVALID;
    // workgroups of a launch are counted in 32 bits
    if ((d->total_q / 128 + d->total_k / 128 + 2 * d->nseq + 2) * d->nheads >= ((int64_t)1 << 31)) return SSD_ERR_UNSUPPORTED;
    const int64_t elem = d->dtype == SSD_BF16 ? 2 : 4;
    if ((rc = check_stride(d->q_stride, d->nheads * d->headdim, elem, p.q_stride)) != SSD_OK) return rc;
    if ((rc = check_stride(d->k_stride, d->nkvheads * d->headdim, elem, p.k_stride)) != SSD_OK) return rc;
    if ((rc = check_stride(d->v_stride, d->nkvheads * d->headdim, elem, p.v_stride)) != SSD_OK) return rc;
    bias = table ? ssd::kBiasBuckets : slopes ? ssd::kBiasSlopes : ssd::kBiasNone;
    if (table && (rc = make_buckets(p.bk, d->num_buckets, d->max_distance, d->bidirectional)) != SSD_OK) return rc;
    if (d->nseq > 0 && ((d->total_q > 0 && !q) || (d->total_k > 0 && (!k || !v)))) return SSD_ERR_INVALID;
    const void* wide[] = {q, k, v, slopes, table};
    for (const void* x : wide)
        if (x && !aligned(x, 16)) return SSD_ERR_ALIGN;
    const void* offsets[] = {cu_q, cu_k, prefix};
    for (const void* x : offsets)
        if (x && !aligned(x, 8)) return SSD_ERR_ALIGN;
    p.q = q;
    p.k = k;
    p.v = v;
    p.slopes = slopes;
    p.table = table;
    p.cu_q = cu_q;
    p.cu_k = cu_k ? cu_k : cu_q;
    p.prefix = prefix;
    p.nseq = d->nseq;
    p.total_q = d->total_q;
    p.total_k = d->total_k;
    p.H = (int)d->nheads;
    p.Hk = (int)d->nkvheads;
    p.causal = d->causal;
    p.scale = d->scale;
    p.cap = take_cap(d->softcap);
    return SSD_OK;
}

// Whether an output is one of the inputs (kernels read inputs after their first stores to outputs) or another output.
template <size_t N, size_t M> bool shared(const void* const (&outputs)[N], const void* const (&inputs)[M]) {
    for (size_t o = 0; o < N; ++o) {
        if (!outputs[o]) continue;
        for (const void* i : inputs)
            if (outputs[o] == i) return true;
        for (size_t i = 0; i < o; ++i)
            if (outputs[o] == outputs[i]) return true;
    }
    return false;
}

int code(int rc) { return rc == 0 ? SSD_OK : rc == -2 ? SSD_ERR_UNSUPPORTED : SSD_ERR_HIP; }

size_t align16(size_t n) { return (n + 15) & ~(size_t)15; }

// Workspace of the backward pass: D per (query, head), the table's partial gradients, and the orders of
// the query and key tiles (twice each: as found and as sorted).  The tiles are bounded without the
// offsets, so that the size does not depend on how a call gives its sequences; table gradients of small
// problems come in tiles of 32 queries, and their key gradients in parts (an equal batch has the fewest
// tiles, and so the most parts).
struct BackwardWorkspace {
    size_t delta, part, dkv, plan_q, plan_k, total;
};
BackwardWorkspace backward_workspace(const ssd_attn_dims* d, bool table) {
    BackwardWorkspace w{};
    const int row_bytes = (int)d->headdim * (d->dtype == SSD_BF16 ? 2 : 4);
    const int64_t q_slots = d->total_q / 128 + d->nseq + 1, k_slots = d->total_k / 128 + d->nseq + 1;
    int64_t parts = q_slots;
    if (d->total_q / 128 * d->nheads < ssd::attn_split_below(row_bytes)) parts = d->total_q / 32 + d->nseq + 1;
    w.delta = align16((size_t)d->total_q * (size_t)d->nheads * 4);
    w.part = table ? align16((size_t)parts * (size_t)d->nheads * (size_t)d->num_buckets * 4) : 0;
    const int n = d->nseq > 0 ? ssd::attn_key_parts(nullptr, d->total_k - d->total_k % d->nseq, d->nseq, d->nkvheads, row_bytes) : 1;
    w.dkv = n > 1 ? align16((size_t)(2 * n) * (size_t)d->total_k * (size_t)d->nkvheads * (size_t)d->headdim * 4) : 0;
    w.plan_q = align16((size_t)(d->total_q * (d->nheads / d->nkvheads) / 128 + d->nseq + 1) * 16);
    w.plan_k = align16((size_t)k_slots * 16);
    w.total = w.delta + w.part + w.dkv + w.plan_q + w.plan_k;
    return w;
}

int check_cache(const ssd_attn_cache* d) {
    if (!d) return SSD_ERR_INVALID;
    const int rc = check_shape(d->nheads, d->nkvheads, d->headdim, d->dtype);
    if (rc != SSD_OK) return rc;
    if (d->nseq < 0 || d->nseq > kMaxTokens || d->num_pages < 0 || d->num_pages >= ((int64_t)1 << 31) || d->page_size < 1 ||
        d->max_pages < 0 || d->max_pages > kMaxTokens)
        return SSD_ERR_INVALID;
    if (d->page_size % 16 != 0 || d->page_size > 65536 || d->max_pages * d->page_size > kMaxTokens) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// Splits of a sequence's keys: enough workgroups for four on each of the 256 CUs, so that short and long
// sequences even out, of at least 128 keys (a block for each wave) at the longest length, and few
// enough that joining them stays small.  A short cache with a workgroup for every other CU or more is not
// split but gets eight waves a workgroup, which saves the join.  Split (with its join) against eight waves, us, 1000 keys, 32/8
// heads, 16 and 32 and 62 sequences (128, 256 and 496 workgroups):
//     bf16  32 wide 11.4/10.2  17.1/14.2  26.4/21.6      64 wide 14.6/11.8  18.9/14.6  28.5/23.5    128 wide 21.7/18.0  28.9/23.1  44.9/42.3
//     fp32  32 wide 15.4/14.1  20.6/16.6  31.8/25.6      64 wide 23.6/21.6  32.5/25.2  50.1/45.7    128 wide 39.1/46.6  64.9/55.8  139/126
// and more at 256 and 512 keys (6 to 40%).  In fp32 at 128 wide eight waves' tiles fill a CU's LDS: there below 256
// workgroups only up to 256 keys (15.4/15.3; 23.3/26.5 at 512).  One sequence: 10.8 split, 15.2 (bf16, 128 wide).
struct DecodeShape {
    int splits, wide;
};
constexpr int64_t kWideKeys = 1024, kWideKeysFullLds = 256;
DecodeShape decode_shape(const ssd_attn_cache* d) {
    const int64_t group = d->nheads / d->nkvheads, units = d->nseq * d->nkvheads * ((group + 15) / 16);
    const int64_t keys = d->max_pages * d->page_size;
    const bool full_lds = d->headdim * (d->dtype == SSD_BF16 ? 2 : 4) >= 512;
    if (keys <= (full_lds && units < 256 ? kWideKeysFullLds : kWideKeys) && units >= 128 && units < 512) return {1, 1};
    int64_t n = units > 0 ? (1024 + units - 1) / units : 1;
    const int64_t most = (keys + 127) / 128;
    if (n > most) n = most;
    if (n > 64) n = 64;
    return {n < 1 ? 1 : (int)n, 0};
}

struct DecodeWorkspace {
    size_t o, ml, total;
};
DecodeWorkspace decode_workspace(const ssd_attn_cache* d) {
    DecodeWorkspace w{};
    const size_t n = (size_t)decode_shape(d).splits, units = (size_t)d->nseq * (size_t)d->nheads;
    if (n > 1) {
        w.o = units * n * (size_t)d->headdim * 4;
        w.ml = align16(units * n * 2 * 4);
    }
    w.total = w.o + w.ml;
    return w;
}

}  // namespace

extern "C" {

int ssd_attn_forward(const ssd_attn_dims* dims, const int64_t* cu_seqlens_q, const int64_t* cu_seqlens_k,
                     const int64_t* prefix, const void* q, const void* k, const void* v, const float* slopes,
                     const float* table, void* y, float* lse, void* stream) {
    ssd::AttnParams p{};
    int bias = 0;
    const int rc = fill(dims, cu_seqlens_q, cu_seqlens_k, prefix, q, k, v, slopes, table, p, bias);
    if (rc != SSD_OK) return rc;
    const bool work = p.nseq > 0 && p.total_q > 0;
    if (work && !y) return SSD_ERR_INVALID;
    if ((y && !aligned(y, 16)) || (lse && !aligned(lse, 16))) return SSD_ERR_ALIGN;
    if (!work) return SSD_OK;
    if (shared({y, lse}, {q, k, v, slopes, table, cu_seqlens_q, cu_seqlens_k, prefix})) return SSD_ERR_INVALID;
    p.y = y;
    p.lse = lse;
    return code(ssd::launch_attn_forward(p, dims->dtype, (int)dims->headdim, bias, static_cast<hipStream_t>(stream)));
}

size_t ssd_attn_backward_workspace_bytes(const ssd_attn_dims* d, int want_dtable) {
    if (!d || d->nseq <= 0 || d->nseq > kMaxTokens || d->total_q < 0 || d->total_q > kMaxTokens || d->total_k < 0 ||
        d->total_k > kMaxTokens || check_shape(d->nheads, d->nkvheads, d->headdim, d->dtype) != SSD_OK ||
        (want_dtable && (d->num_buckets < 2 || d->num_buckets > 2 * ssd::kMaxBorders)))
        return 0;
    return backward_workspace(d, want_dtable != 0).total;
}

int ssd_attn_backward(const ssd_attn_dims* dims, const int64_t* cu_seqlens_q, const int64_t* cu_seqlens_k,
                      const int64_t* prefix, const void* q, const void* k, const void* v, const float* slopes,
                      const float* table, const void* y, const float* lse, const void* dy, void* dq, void* dk, void* dv,
                      float* dtable, void* workspace, size_t workspace_bytes, void* stream) {
    ssd::AttnParams p{};
    int bias = 0;
    const int rc = fill(dims, cu_seqlens_q, cu_seqlens_k, prefix, q, k, v, slopes, table, p, bias);
    if (rc != SSD_OK) return rc;
    if (dtable && !table) return SSD_ERR_INVALID;
    const bool queries = p.nseq > 0 && p.total_q > 0, keys = p.nseq > 0 && p.total_k > 0;
    if ((queries && (!y || !lse || !dy || !dq)) || (keys && (!dk || !dv))) return SSD_ERR_INVALID;
    const void* wide[] = {y, lse, dy, dq, dk, dv, dtable, workspace};
    for (const void* x : wide)
        if (x && !aligned(x, 16)) return SSD_ERR_ALIGN;
    const BackwardWorkspace w = backward_workspace(dims, dtable != nullptr);
    if (p.nseq > 0 && w.total > 0 && (!workspace || workspace_bytes < w.total)) return SSD_ERR_INVALID;
    if (!queries && !keys && !dtable) return SSD_OK;
    if (shared({dq, dk, dv, dtable, workspace}, {q, k, v, y, lse, dy, slopes, table, cu_seqlens_q, cu_seqlens_k, prefix}))
        return SSD_ERR_INVALID;
    p.y = const_cast<void*>(y);
    p.lse = const_cast<float*>(lse);
    p.dy = dy;
    p.dq = dq;
    p.dk = dk;
    p.dv = dv;
    p.dtable = dtable;
    p.delta = static_cast<float*>(workspace);
    char* at = static_cast<char*>(workspace) + w.delta;
    p.table_part = dtable ? reinterpret_cast<float*>(at) : nullptr;
    p.dkv_part = w.dkv > 0 ? reinterpret_cast<float*>(at + w.part) : nullptr;
    if (p.cu_q && p.nseq > 1) {
        p.plan_q = reinterpret_cast<int2*>(at + w.part + w.dkv);
        p.plan_k = reinterpret_cast<int2*>(at + w.part + w.dkv + w.plan_q);
    }
    return code(ssd::launch_attn_backward(p, dims->dtype, (int)dims->headdim, bias, static_cast<hipStream_t>(stream)));
}

size_t ssd_attn_decode_workspace_bytes(const ssd_attn_cache* d) {
    return check_cache(d) == SSD_OK ? decode_workspace(d).total : 0;
}

int ssd_attn_decode(const ssd_attn_cache* d, const void* q, const void* k_cache, const void* v_cache,
                    const int32_t* block_table, const int64_t* seq_lens, const float* slopes, const float* table, void* y,
                    void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_cache(d);
    if (rc != SSD_OK) return rc;
    if (!std::isfinite(d->scale) || !std::isfinite(d->softcap) || d->softcap < 0.f || (slopes && table)) return SSD_ERR_INVALID;
    ssd::DecodeParams p{};
    if ((rc = check_stride(d->q_stride, d->nheads * d->headdim, d->dtype == SSD_BF16 ? 2 : 4, p.q_stride)) != SSD_OK) return rc;
    if (table && (rc = make_buckets(p.bk, d->num_buckets, d->max_distance, d->bidirectional)) != SSD_OK) return rc;
    const bool cached = d->num_pages > 0 && d->max_pages > 0;
    if (d->nseq > 0 && (!q || !y || !seq_lens || (cached && (!k_cache || !v_cache)) || (d->max_pages > 0 && !block_table)))
        return SSD_ERR_INVALID;
    const void* wide[] = {q, k_cache, v_cache, slopes, table, y, workspace};
    for (const void* x : wide)
        if (x && !aligned(x, 16)) return SSD_ERR_ALIGN;
    if ((block_table && !aligned(block_table, 4)) || (seq_lens && !aligned(seq_lens, 8))) return SSD_ERR_ALIGN;
    const DecodeShape shape = decode_shape(d);
    p.splits = shape.splits;
    p.wide = shape.wide;
    if (d->nseq * d->nheads * p.splits >= ((int64_t)1 << 31)) return SSD_ERR_UNSUPPORTED;
    const DecodeWorkspace w = decode_workspace(d);
    if (w.total > 0 && (!workspace || workspace_bytes < w.total)) return SSD_ERR_INVALID;
    if (d->nseq == 0) return SSD_OK;
    if (shared({y, workspace}, {q, k_cache, v_cache, block_table, seq_lens, slopes, table})) return SSD_ERR_INVALID;
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.slopes = slopes;
    p.table = table;
    p.y = y;
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = w.total > 0 ? reinterpret_cast<float*>(static_cast<char*>(workspace) + w.o) : nullptr;
    p.nseq = d->nseq;
    p.H = (int)d->nheads;
    p.Hk = (int)d->nkvheads;
    p.num_pages = (int)d->num_pages;
    p.page_size = (int)d->page_size;
    p.max_pages = (int)d->max_pages;
    p.scale = d->scale;
    p.cap = take_cap(d->softcap);
    const int bias = table ? ssd::kBiasBuckets : slopes ? ssd::kBiasSlopes : ssd::kBiasNone;
    return code(ssd::launch_attn_decode(p, d->dtype, (int)d->headdim, bias, static_cast<hipStream_t>(stream)));
}

int ssd_kv_append(const ssd_attn_cache* d, int64_t tokens, const int64_t* cu_seqlens, const int64_t* seq_lens,
                  const int32_t* block_table, const void* k, const void* v, const void* q, const float* inv_freq,
                  int rot_pairs, int interleaved, void* k_cache, void* v_cache, void* q_out, void* stream) {
    int rc = check_cache(d);
    if (rc != SSD_OK) return rc;
    if (tokens < 0 || tokens > kMaxTokens || (!cu_seqlens && tokens != d->nseq)) return SSD_ERR_INVALID;
    if ((interleaved != 0 && interleaved != 1) || rot_pairs < 0 || 2 * (int64_t)rot_pairs > d->headdim || (rot_pairs > 0 && !inv_freq))
        return SSD_ERR_INVALID;
    if (rot_pairs % 8 != 0) return SSD_ERR_UNSUPPORTED;
    ssd::AppendParams p{};
    const int64_t elem = d->dtype == SSD_BF16 ? 2 : 4;
    if ((rc = check_stride(d->q_stride, d->nheads * d->headdim, elem, p.q_stride)) != SSD_OK) return rc;
    if ((rc = check_stride(d->k_stride, d->nkvheads * d->headdim, elem, p.k_stride)) != SSD_OK) return rc;
    if ((rc = check_stride(d->v_stride, d->nkvheads * d->headdim, elem, p.v_stride)) != SSD_OK) return rc;
    if (!q != !q_out) return SSD_ERR_INVALID;
    const bool cached = d->num_pages > 0 && d->max_pages > 0;
    if (tokens > 0 && d->nseq > 0 &&
        (!k || !v || !seq_lens || (cached && (!k_cache || !v_cache)) || (d->max_pages > 0 && !block_table)))
        return SSD_ERR_INVALID;
    const void* wide[] = {q, k, v, q_out, k_cache, v_cache, inv_freq};
    for (const void* x : wide)
        if (x && !aligned(x, 16)) return SSD_ERR_ALIGN;
    if ((block_table && !aligned(block_table, 4)) || (seq_lens && !aligned(seq_lens, 8)) || (cu_seqlens && !aligned(cu_seqlens, 8)))
        return SSD_ERR_ALIGN;
    if (tokens == 0 || d->nseq == 0) return SSD_OK;
    if (shared({k_cache, v_cache, q_out}, {k, v, q, cu_seqlens, seq_lens, block_table, inv_freq})) return SSD_ERR_INVALID;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_out = q_out;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.cu = cu_seqlens;
    p.inv_freq = inv_freq;
    p.nseq = d->nseq;
    p.tokens = tokens;
    p.H = (int)d->nheads;
    p.Hk = (int)d->nkvheads;
    p.D = (int)d->headdim;
    p.num_pages = (int)d->num_pages;
    p.page_size = (int)d->page_size;
    p.max_pages = (int)d->max_pages;
    p.rot = inv_freq ? rot_pairs : 0;
    p.interleaved = interleaved;
    return code(ssd::launch_kv_append(p, d->dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
