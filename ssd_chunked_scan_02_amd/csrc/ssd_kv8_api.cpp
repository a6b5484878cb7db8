// C ABI of the 8-bit paged cache and of the rotation (declared in include/ssd_kv8.h and include/ssd_rotary.h): argument
// validation, workspace sizing and dispatch to the kernels.  Every check runs before the first HIP call.
#include "ssd_kv8.h"
#include "ssd_rotary.h"

#include <cmath>

#include <hip/hip_runtime.h>

#include "ssd_attn_checks.h"
#include "ssd_kv8_launch.h"

namespace {

using namespace ssd::checks;

int64_t elem_of(const ssd_attn_cache* d) { return d->dtype == SSD_BF16 ? 2 : 4; }

// The pages of a call, their pointers needed where there is anything they could hold.
int take_pages(const ssd_attn_cache* d, const ssd_kv8_pages* g, bool needed, ssd::Kv8Pages& out) {
    if (!g || (g->format != SSD_KV8_INT8 && g->format != SSD_KV8_E4M3)) return SSD_ERR_INVALID;
    if (needed && d->num_pages > 0 && d->max_pages > 0 && any_null({g->k, g->v, g->k_scale, g->v_scale})) return SSD_ERR_INVALID;
    if (!all_aligned({g->k, g->v, g->k_scale, g->v_scale}, 16)) return SSD_ERR_ALIGN;
    out = ssd::Kv8Pages{static_cast<uint8_t*>(g->k), static_cast<uint8_t*>(g->v), g->k_scale, g->v_scale};
    return SSD_OK;
}

// As decode_shape, on this kernel's own times.  Its tiles of values are bf16 for either type of the queries (8.7 KB a wave at 128
// wide), and a cache of 128 keys or fewer, which is not split either way, has too few blocks for eight waves.  Split (with its join)
// against eight waves, us, 32/8 heads, int8, of 256 and 1000 keys, by workgroups (key heads of all sequences):
//                    64                   96                   128                  256                   496                   640
//     bf16  64 wide  7.3/6.3 11.1/12.1    7.4/6.4 12.4/12.1    7.5/6.3 13.4/12.1    8.9/6.5 16.5/13.5     11.1/8.6 25.2/19.9    12.7/12.1 27.4/27.2
//          128 wide  9.0/8.4 13.4/16.4    9.0/8.5 16.3/17.7    9.0/8.5 19.6/17.7    11.5/8.7 24.5/19.5    17.4/16.6 36.9/34.7   20.3/23.9 40.3/48.6
//     fp32  64 wide  7.8/6.8 11.7/13.1    7.8/6.9 13.3/13.2    7.8/6.9 15.4/13.2    9.5/7.0 19.4/15.0     12.8/12.1 28.8/27.4   15.1/17.6 31.8/38.6
//          128 wide  9.7/9.4 14.6/18.5    9.7/9.5 19.8/19.8    9.8/9.5 22.7/19.8    12.5/9.6 29.1/21.6    20.7/19.1 44.5/39.3   24.8/27.4 49.7/55.0
// 2000 keys: 18.1/21.3 and 25.9/29.4 (bf16, 128 workgroups, 64 and 128 wide); 128 keys: 8.6/11.8 (bf16, 128 wide, 496).  e4m3: the
// same sides, up to 10% less.
DecodeShape kv8_shape(const ssd_attn_cache* d) {
    const int64_t units = decode_units(d), keys = d->max_pages * d->page_size;
    if (keys > 128 && keys <= kWideKeys && units >= 128 && units < 512) return {1, 1};
    return split_shape(units, keys);
}

struct Kv8Workspace {
    size_t o, ml, total;
};
Kv8Workspace decode_workspace(const ssd_attn_cache* d) {
    Kv8Workspace w{};
    const size_t n = (size_t)kv8_shape(d).splits, units = (size_t)d->nseq * (size_t)d->nheads;
    if (n > 1) {
        w.o = units * n * (size_t)d->headdim * 4;
        w.ml = align16(units * n * 2 * 4);
    }
    w.total = w.o + w.ml;
    return w;
}

}  // namespace

extern "C" {

int ssd_kv8_append(const ssd_attn_cache* d, const ssd_kv8_pages* pages, int64_t tokens, const int64_t* cu_seqlens,
                   const int64_t* seq_lens, const int32_t* block_table, const void* k, const void* v, const void* q,
                   const float* inv_freq, int rot_pairs, int interleaved, void* q_out, void* stream) {
    int rc = check_cache(d);
    if (rc != SSD_OK) return rc;
    if (tokens < 0 || tokens > kMaxTokens || (!cu_seqlens && tokens != d->nseq)) return SSD_ERR_INVALID;
    if ((interleaved != 0 && interleaved != 1) || rot_pairs < 0 || 2 * (int64_t)rot_pairs > d->headdim || (rot_pairs > 0 && !inv_freq))
        return SSD_ERR_INVALID;
    if (rot_pairs % 8 != 0) return SSD_ERR_UNSUPPORTED;
    ssd::AppendParams p{};
    ssd::Kv8Pages g{};
    if ((rc = stride(d->q_stride, d->nheads * d->headdim, elem_of(d), p.q_stride)) != SSD_OK) return rc;
    if ((rc = stride(d->k_stride, d->nkvheads * d->headdim, elem_of(d), p.k_stride)) != SSD_OK) return rc;
    if ((rc = stride(d->v_stride, d->nkvheads * d->headdim, elem_of(d), p.v_stride)) != SSD_OK) return rc;
    const bool work = tokens > 0 && d->nseq > 0;
    if ((rc = take_pages(d, pages, work, g)) != SSD_OK) return rc;
    if (!q != !q_out) return SSD_ERR_INVALID;
    if (work && (any_null({k, v, seq_lens}) || (d->max_pages > 0 && !block_table))) return SSD_ERR_INVALID;
    if (!all_aligned({q, k, v, q_out, inv_freq}, 16) || !aligned(block_table, 4) || !all_aligned({seq_lens, cu_seqlens}, 8)) return SSD_ERR_ALIGN;
    if (!work) return SSD_OK;
    if (shared({pages->k, pages->v, pages->k_scale, pages->v_scale, q_out}, {k, v, q, cu_seqlens, seq_lens, block_table, inv_freq}))
        return SSD_ERR_INVALID;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_out = q_out;
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
    return code(ssd::launch_kv8_append(p, g, d->dtype, pages->format, static_cast<hipStream_t>(stream)));
}

size_t ssd_kv8_decode_workspace_bytes(const ssd_attn_cache* d) { return check_cache(d) == SSD_OK ? decode_workspace(d).total : 0; }

int ssd_kv8_decode(const ssd_attn_cache* d, const ssd_kv8_pages* pages, const void* q, const int32_t* block_table,
                   const int64_t* seq_lens, const float* slopes, const float* table, void* y, void* workspace,
                   size_t workspace_bytes, void* stream) {
    int rc = check_cache(d);
    if (rc != SSD_OK) return rc;
    if (!std::isfinite(d->scale) || !std::isfinite(d->softcap) || d->softcap < 0.f || (slopes && table)) return SSD_ERR_INVALID;
    ssd::DecodeParams p{};
    ssd::Kv8Pages g{};
    if ((rc = stride(d->q_stride, d->nheads * d->headdim, elem_of(d), p.q_stride)) != SSD_OK) return rc;
    if (table && (rc = make_buckets(p.bk, d->num_buckets, d->max_distance, d->bidirectional)) != SSD_OK) return rc;
    if ((rc = take_pages(d, pages, d->nseq > 0, g)) != SSD_OK) return rc;
    if (d->nseq > 0 && (any_null({q, y, seq_lens}) || (d->max_pages > 0 && !block_table))) return SSD_ERR_INVALID;
    if (!all_aligned({q, slopes, table, y, workspace}, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 8)) return SSD_ERR_ALIGN;
    const DecodeShape shape = kv8_shape(d);
    p.splits = shape.splits;
    p.wide = shape.wide;
    if (d->nseq * d->nheads * p.splits >= ((int64_t)1 << 31)) return SSD_ERR_UNSUPPORTED;
    const Kv8Workspace w = decode_workspace(d);
    if (w.total > 0 && (!workspace || workspace_bytes < w.total)) return SSD_ERR_INVALID;
    if (d->nseq == 0) return SSD_OK;
    if (shared({y, workspace}, {q, pages->k, pages->v, pages->k_scale, pages->v_scale, block_table, seq_lens, slopes, table})) return SSD_ERR_INVALID;
    p.q = q;
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
    return code(ssd::launch_kv8_decode(p, g, d->dtype, pages->format, (int)d->headdim, bias, static_cast<hipStream_t>(stream)));
}

int ssd_kv8_read(const ssd_attn_cache* d, const ssd_kv8_pages* pages, int64_t tokens, const int64_t* cu_seqlens,
                 const int64_t* seq_lens, const int32_t* block_table, void* k, void* v, void* stream) {
    int rc = check_cache(d);
    if (rc != SSD_OK) return rc;
    if (tokens < 0 || tokens > kMaxTokens || (!cu_seqlens && d->nseq > 0 && tokens % d->nseq != 0)) return SSD_ERR_INVALID;
    ssd::Kv8ReadParams p{};
    const bool work = tokens > 0 && d->nseq > 0;
    if ((rc = take_pages(d, pages, work, p.pages)) != SSD_OK) return rc;
    if (work && (any_null({k, v, seq_lens}) || (d->max_pages > 0 && !block_table))) return SSD_ERR_INVALID;
    if (!all_aligned({k, v}, 16) || !aligned(block_table, 4) || !all_aligned({seq_lens, cu_seqlens}, 8)) return SSD_ERR_ALIGN;
    if (!work) return SSD_OK;
    if (shared({k, v}, {pages->k, pages->v, pages->k_scale, pages->v_scale, cu_seqlens, seq_lens, block_table})) return SSD_ERR_INVALID;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.cu = cu_seqlens;
    p.k = k;
    p.v = v;
    p.nseq = d->nseq;
    p.tokens = tokens;
    p.each = tokens / d->nseq;
    p.Hk = (int)d->nkvheads;
    p.D = (int)d->headdim;
    p.num_pages = (int)d->num_pages;
    p.page_size = (int)d->page_size;
    p.max_pages = (int)d->max_pages;
    return code(ssd::launch_kv8_read(p, d->dtype, pages->format, static_cast<hipStream_t>(stream)));
}

int ssd_rotate(const ssd_rotary_dims* d, const int64_t* cu_seqlens, const int64_t* start, const void* q, const void* k,
               const float* inv_freq, void* q_out, void* k_out, void* stream) {
    if (!d) return SSD_ERR_INVALID;
    if (d->nseq < 0 || d->nseq > kMaxTokens || d->total < 0 || d->total > kMaxTokens || d->nheads < 1 || d->nheads > kMaxHeads || d->headdim < 1)
        return SSD_ERR_INVALID;
    if (d->dtype != SSD_F32 && d->dtype != SSD_BF16) return SSD_ERR_INVALID;
    if ((d->interleaved != 0 && d->interleaved != 1) || (d->inverse != 0 && d->inverse != 1) || !std::isfinite(d->magnitude)) return SSD_ERR_INVALID;
    if (d->rot_pairs < 0 || 2 * (int64_t)d->rot_pairs > d->headdim || (d->rot_pairs > 0 && !inv_freq)) return SSD_ERR_INVALID;
    if (!k != !k_out || (k && (d->nkvheads < 1 || d->nkvheads > kMaxHeads))) return SSD_ERR_INVALID;
    if (d->nseq > 0 && !cu_seqlens && d->total % d->nseq != 0) return SSD_ERR_INVALID;
    const int64_t D = d->headdim;
    if ((D != 32 && D != 64 && D != 128) || d->rot_pairs % 8 != 0) return SSD_ERR_UNSUPPORTED;
    if (d->nheads * D >= ((int64_t)1 << 24) || (k && d->nkvheads * D >= ((int64_t)1 << 24))) return SSD_ERR_UNSUPPORTED;
    ssd::RotateParams p{};
    const int64_t elem = d->dtype == SSD_BF16 ? 2 : 4;
    int rc = stride(d->q_stride, d->nheads * D, elem, p.q_stride);
    if (rc == SSD_OK && k) rc = stride(d->k_stride, d->nkvheads * D, elem, p.k_stride);
    if (rc != SSD_OK) return rc;
    const bool work = d->nseq > 0 && d->total > 0;
    if (work && any_null({q, q_out})) return SSD_ERR_INVALID;
    if (!all_aligned({q, k, q_out, k_out, inv_freq}, 16) || !all_aligned({cu_seqlens, start}, 8)) return SSD_ERR_ALIGN;
    if (!work) return SSD_OK;
    if (shared({q_out, k_out}, {q, k, inv_freq, cu_seqlens, start})) return SSD_ERR_INVALID;
    p.q = q;
    p.k = k;
    p.q_out = q_out;
    p.k_out = k_out;
    p.cu = cu_seqlens;
    p.start = start;
    p.inv_freq = inv_freq;
    p.nseq = d->nseq;
    p.total = d->total;
    p.each = d->total / d->nseq;
    p.H = (int)d->nheads;
    p.Hk = k ? (int)d->nkvheads : 0;
    p.D = (int)D;
    p.rot = inv_freq ? d->rot_pairs : 0;
    p.interleaved = d->interleaved;
    p.magnitude = d->magnitude;
    p.sign = d->inverse ? -1.f : 1.f;
    return code(ssd::launch_rotate(p, d->dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
