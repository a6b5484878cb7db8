// C ABI of the gated delta rule (declared in include/ssd_delta.h): argument validation, workspace layout and dispatch
// to the kernels.  Every check runs before the first HIP call.
#include "ssd_delta.h"

#include <cmath>

#include <hip/hip_runtime.h>

#include "ssd_checks.h"
#include "ssd_delta_launch.h"

namespace {

using namespace ssd::checks;

int check_dims(const ssd_delta_dims* d, bool step) {
    if (!d) return SSD_ERR_INVALID;
    if (d->nheads < 1 || d->ngroups < 1 || d->nheads > kMaxHeads || d->nheads % d->ngroups != 0 || d->keydim < 1 || d->valuedim < 1)
        return SSD_ERR_INVALID;
    if (d->dtype != SSD_F32 && d->dtype != SSD_BF16) return SSD_ERR_INVALID;
    if (d->nseq < 0 || d->nseq > kMaxTokens || (!step && (d->total < 0 || d->total > kMaxTokens))) return SSD_ERR_INVALID;
    if (!std::isfinite(d->scale)) return SSD_ERR_INVALID;
    if ((d->keydim != 32 && d->keydim != 64 && d->keydim != 128) || d->valuedim % ssd::kDeltaCols != 0 || d->valuedim > 256)
        return SSD_ERR_UNSUPPORTED;
    if (d->ngroups * d->keydim >= ((int64_t)1 << 24) || d->nheads * d->valuedim >= ((int64_t)1 << 24)) return SSD_ERR_UNSUPPORTED;
    const int64_t walks = d->nseq * d->nheads * (d->valuedim / 16) + 8;
    const int64_t chunks = step ? 0 : ssd::delta_slots(d->total, d->nseq) * d->ngroups;
    if (!launchable(walks, 256) || !launchable(chunks, 512)) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

int strides(const ssd_delta_dims* d, int64_t& q, int64_t& k, int64_t& v) {
    const int64_t elem = d->dtype == SSD_BF16 ? 2 : 4;
    int rc = stride(d->q_stride, d->ngroups * d->keydim, elem, q);
    if (rc == SSD_OK) rc = stride(d->k_stride, d->ngroups * d->keydim, elem, k);
    if (rc == SSD_OK) rc = stride(d->v_stride, d->nheads * d->valuedim, elem, v);
    return rc;
}

// Columns of a walk's workgroup.  With 32 each load of K, Q, Z and the scores serves twice the columns, with 16 the steps
// of a chunk are shorter: 16 where its workgroups still have one of the 256 CUs each.  Forward and training step of one
// sequence of 2048 tokens, us, 16 against 32 columns:
//     bf16, 64 by 64     128 workgroups of 16 72/287 against 91/359, 256: 86/419 against 101/462, 384: 133/639 against 120/553
//     bf16, 128 by 128   128: 78/316 against 102/426, 256: 94/446 against 111/522, 384: 125/669 against 118/597
//     fp32, 64 by 64     128: 97/379 against 135/501, 256: 123/525 against 156/638, 384: 192/812 against 176/764
//     fp32, 128 by 128   128: 127/495 against 199/723, 256: 151/654 against 217/872, 384: 234/1077 against 233/993
// and of four sequences with 768 and 1024 workgroups of 16, bf16, 128 by 64: 314/1447 against 283/1294, 395/1871 against 337/1570.
int walk_columns(const ssd_delta_dims* d) { return d->nseq * d->nheads * (d->valuedim / 16) <= 256 ? 16 : 32; }

// Lays the workspace out from `base` (null: only its size is wanted), and returns its bytes.
size_t lay_out(const ssd_delta_dims* d, bool backward, char* base, ssd::DeltaParams& p) {
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        char* here = base ? base + at : nullptr;
        at += align16(bytes);
        return here;
    };
    const size_t elem = d->dtype == SSD_BF16 ? 2 : 4, terms = d->dtype == SSD_BF16 ? 3 : 1;
    const size_t slots = (size_t)ssd::delta_slots(d->total, d->nseq), H = (size_t)d->nheads, G = (size_t)d->ngroups;
    const size_t N = (size_t)d->keydim, P = (size_t)d->valuedim, C = ssd::kDeltaChunk, blocks = P / (size_t)walk_columns(d);
    if (d->total == 0 || d->nseq == 0) return 0;
    p.z = take(slots * H * terms * C * C * elem);
    p.scores = take(slots * H * (backward || terms == 1 ? terms : 2) * C * C * elem);
    const size_t walked = at;  // what the walk down the chunks alone reads
    p.kr = take(slots * G * N * C * elem);
    p.qr = take(slots * G * N * C * elem);
    p.gates = reinterpret_cast<float*>(take(slots * H * ssd::kDeltaGates * C * 4));
    if (!backward) return at;
    p.zt = take(slots * H * terms * C * C * elem);
    p.scores_t = take(slots * H * terms * C * C * elem);
    p.states = reinterpret_cast<float*>(take((slots + (size_t)d->nseq) * H * N * P * 4));
    p.wrong = reinterpret_cast<float*>(take((size_t)d->total * H * P * 4));
    p.dstates = take(slots * H * N * P * elem);
    if (terms > 1) {
        // in the place of Z and the scores, which the backward walk does not read, where there is room (N P + 64 P of 24576
        // elements for a chunk and head: all but keys of 128 with values of 160 and more)
        const size_t states = align16(slots * H * N * P * elem), values = align16((size_t)d->total * H * P * elem);
        const bool room = states + values <= walked;
        p.dstates_rest = room ? base : take(states);
        p.dv_rest = room ? (base ? base + states : nullptr) : take(values);
    }
    p.dot_y = reinterpret_cast<float*>(take(slots * H * blocks * C * 4));
    p.dot_v = reinterpret_cast<float*>(take(slots * H * blocks * C * 4));
    p.dot_b = reinterpret_cast<float*>(take(slots * H * blocks * C * 4));
    p.dot_s = reinterpret_cast<float*>(take(slots * H * blocks * 4 * 4));
    p.dot_0 = reinterpret_cast<float*>(take((size_t)d->nseq * H * blocks * 4 * 4));
    return at;
}

// What both passes check alike; fills their shared launch parameters.
int fill(const ssd_delta_dims* d, const int64_t* cu, const void* q, const void* k, const void* v, const float* log_a,
         const float* beta, const float* init, bool backward, void* workspace, size_t workspace_bytes, ssd::DeltaParams& p) {
    int rc = check_dims(d, false);
    if (rc == SSD_OK) rc = strides(d, p.q_stride, p.k_stride, p.v_stride);
    if (rc != SSD_OK) return rc;
    if (d->nseq > 0 && !cu && d->total % d->nseq != 0) return SSD_ERR_INVALID;
    if (d->nseq > 0 && d->total > 0 && any_null({q, k, v, log_a, beta})) return SSD_ERR_INVALID;
    if (!all_aligned({q, k, v, log_a, beta, init, workspace}, 16) || !aligned(cu, 8)) return SSD_ERR_ALIGN;
    const size_t need = lay_out(d, backward, static_cast<char*>(workspace), p);
    if (need > 0 && (!workspace || workspace_bytes < need)) return SSD_ERR_INVALID;
    p.q = q;
    p.k = k;
    p.v = v;
    p.log_a = log_a;
    p.beta = beta;
    p.init = init;
    p.cu = cu;
    p.nseq = d->nseq;
    p.total = d->total;
    p.each = d->nseq > 0 ? d->total / d->nseq : 0;
    p.slots = ssd::delta_slots(d->total, d->nseq);
    p.H = (int)d->nheads;
    p.G = (int)d->ngroups;
    p.N = (int)d->keydim;
    p.P = (int)d->valuedim;
    p.cols = walk_columns(d);
    p.scale = d->scale;
    return SSD_OK;
}

size_t workspace_bytes_of(const ssd_delta_dims* d, bool backward) {
    ssd::DeltaParams p{};
    return check_dims(d, false) == SSD_OK ? lay_out(d, backward, nullptr, p) : 0;
}

}  // namespace

extern "C" {

size_t ssd_delta_forward_workspace_bytes(const ssd_delta_dims* d) { return workspace_bytes_of(d, false); }

int ssd_delta_forward(const ssd_delta_dims* d, const int64_t* cu_seqlens, const void* q, const void* k, const void* v,
                      const float* log_a, const float* beta, const float* init_state, void* y, float* final_state,
                      void* workspace, size_t workspace_bytes, void* stream) {
    ssd::DeltaParams p{};
    const int rc = fill(d, cu_seqlens, q, k, v, log_a, beta, init_state, false, workspace, workspace_bytes, p);
    if (rc != SSD_OK) return rc;
    const bool tokens = p.nseq > 0 && p.total > 0;
    if (tokens && !y) return SSD_ERR_INVALID;
    if (!all_aligned({y, final_state}, 16)) return SSD_ERR_ALIGN;
    if (!tokens && (p.nseq == 0 || !final_state)) return SSD_OK;
    if (shared({y, final_state, workspace}, {q, k, v, log_a, beta, cu_seqlens}) || (init_state && (y == init_state || workspace == init_state)))
        return SSD_ERR_INVALID;
    p.y = y;
    p.final_state = final_state;
    return code(ssd::launch_delta_forward(p, d->dtype, static_cast<hipStream_t>(stream)));
}

size_t ssd_delta_backward_workspace_bytes(const ssd_delta_dims* d) { return workspace_bytes_of(d, true); }

int ssd_delta_backward(const ssd_delta_dims* d, const int64_t* cu_seqlens, const void* q, const void* k, const void* v,
                       const float* log_a, const float* beta, const float* init_state, const void* dy, const float* dfinal,
                       void* dq, void* dk, void* dv, float* dlog_a, float* dbeta, float* dinit, void* workspace,
                       size_t workspace_bytes, void* stream) {
    ssd::DeltaParams p{};
    const int rc = fill(d, cu_seqlens, q, k, v, log_a, beta, init_state, true, workspace, workspace_bytes, p);
    if (rc != SSD_OK) return rc;
    const bool tokens = p.nseq > 0 && p.total > 0;
    if (tokens && any_null({dy, dq, dk, dv, dlog_a, dbeta})) return SSD_ERR_INVALID;
    if (!all_aligned({dy, dfinal, dq, dk, dv, dlog_a, dbeta, dinit}, 16)) return SSD_ERR_ALIGN;
    if (!tokens && (p.nseq == 0 || !dinit)) return SSD_OK;
    if (shared({dq, dk, dv, dlog_a, dbeta, dinit, workspace}, {q, k, v, log_a, beta, cu_seqlens, init_state, dy, dfinal}))
        return SSD_ERR_INVALID;
    p.dy = dy;
    p.dfinal = dfinal;
    p.dq = dq;
    p.dk = dk;
    p.dv = dv;
    p.dlog_a = dlog_a;
    p.dbeta = dbeta;
    p.dinit = dinit;
    return code(ssd::launch_delta_backward(p, d->dtype, static_cast<hipStream_t>(stream)));
}

int ssd_delta_step(const ssd_delta_dims* d, float* state, const void* q, const void* k, const void* v, const float* log_a,
                   const float* beta, void* y, void* stream) {
    int rc = check_dims(d, true);
    ssd::DeltaStepParams p{};
    if (rc == SSD_OK) rc = strides(d, p.q_stride, p.k_stride, p.v_stride);
    if (rc != SSD_OK) return rc;
    if (d->nseq > 0 && any_null({state, q, k, v, log_a, beta, y})) return SSD_ERR_INVALID;
    if (!all_aligned({state, q, k, v, log_a, beta, y}, 16)) return SSD_ERR_ALIGN;
    if (d->nseq == 0) return SSD_OK;
    if (shared({state, y}, {q, k, v, log_a, beta})) return SSD_ERR_INVALID;
    p.state = state;
    p.q = q;
    p.k = k;
    p.v = v;
    p.log_a = log_a;
    p.beta = beta;
    p.y = y;
    p.nseq = d->nseq;
    p.H = (int)d->nheads;
    p.G = (int)d->ngroups;
    p.N = (int)d->keydim;
    p.P = (int)d->valuedim;
    p.scale = d->scale;
    return code(ssd::launch_delta_step(p, d->dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
