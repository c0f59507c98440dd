// rotary_api.hip -- the C ABI of the rotary positions and the query and key
// norms declared in include/gdn2.h: host-side validation, then dispatch to the
// gfx950 kernels on the caller's stream.  Validation never touches the GPU.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "api_check.h"
#include "gdn2.h"
#include "linear.h"
#include "rotary.h"

namespace {

using namespace gdn2::api;
using gdn2::RotaryArgs;

gdn2_status check(const gdn2_rotary_desc *d, bool norm) {
    if (!d) return GDN2_ERR_NULL;
    if (d->tokens < 0 || d->period < 1 || d->tokens % d->period != 0 || d->q_heads < 1 || d->k_heads < 0 || d->dim < 1 ||
        d->rotary < 0 || d->rotary > d->dim || d->rotary % 2 != 0)
        return GDN2_ERR_SHAPE;
    if ((d->dtype != GDN2_F32 && d->dtype != GDN2_BF16) || (d->weight_dtype != GDN2_F32 && d->weight_dtype != GDN2_BF16))
        return GDN2_ERR_DTYPE;
    if (d->layout != GDN2_ROTARY_HALF && d->layout != GDN2_ROTARY_INTERLEAVED) return GDN2_ERR_SHAPE;
    if (norm ? d->norm != GDN2_QK_RMS && d->norm != GDN2_QK_L2 : d->norm != GDN2_QK_NONE) return GDN2_ERR_SHAPE;
    if (!(d->eps >= 0.f) || std::isinf(d->eps) || !std::isfinite(d->magnitude)) return GDN2_ERR_SHAPE;
    if (d->offset > (INT64_C(1) << 40) || d->offset < -(INT64_C(1) << 40)) return GDN2_ERR_SHAPE;
    if (d->dim > 256 || d->q_heads > 65535 || d->k_heads > 65535 || d->tokens > INT32_MAX || d->period > INT32_MAX)
        return GDN2_ERR_UNSUPPORTED;
    if (d->q_stride < d->q_heads * d->dim || d->k_stride < d->k_heads * d->dim || !product_ok({d->tokens, d->q_stride, 16}) ||
        !product_ok({d->tokens, d->k_stride, 16}))
        return GDN2_ERR_SHAPE;
    return GDN2_OK;
}

int64_t esize(const gdn2_rotary_desc *d) { return d->dtype == GDN2_BF16 ? 2 : 4; }

// bytes from the first to the last element that a strided / contiguous tensor holds
int64_t strided_bytes(const gdn2_rotary_desc *d, int64_t heads, int64_t stride) {
    return heads && d->tokens ? ((d->tokens - 1) * stride + heads * d->dim) * esize(d) : 0;
}
int64_t dense_bytes(const gdn2_rotary_desc *d, int64_t heads) { return d->tokens * heads * d->dim * esize(d); }

RotaryArgs args_of(const gdn2_rotary_desc *d, const double *freq, const int32_t *positions) {
    RotaryArgs a = {};
    a.freq = freq;
    a.pos = positions;
    a.offset = d->offset;
    a.tokens = static_cast<int>(d->tokens);
    a.period = static_cast<int>(d->period);
    a.d = static_cast<int>(d->dim);
    a.rot = static_cast<int>(d->rotary);
    a.part[0].H = static_cast<int>(d->q_heads);
    a.part[1].H = static_cast<int>(d->k_heads);
    a.part[0].stride = d->q_stride;
    a.part[1].stride = d->k_stride;
    a.bf16 = d->dtype == GDN2_BF16;
    a.w_bf16 = d->weight_dtype == GDN2_BF16;
    a.inter = d->layout == GDN2_ROTARY_INTERLEAVED;
    a.l2 = d->norm == GDN2_QK_L2;
    a.eps = d->eps;
    a.cos_mag = a.sin_mag = d->magnitude;
    return a;
}

// Rotation with or without norm, one input row to one output row.
gdn2_status forward(const gdn2_rotary_desc *d, bool norm, bool back, const void *q, const void *k, const void *qw,
                    const void *kw, const double *freq, const int32_t *positions, void *q_out, void *k_out, void *stream) {
    const gdn2_status st = check(d, norm);
    if (st != GDN2_OK) return st;
    if (d->tokens == 0) return GDN2_OK;
    if (!q || !q_out || (d->k_heads && (!k || !k_out)) || (d->rotary && !freq)) return GDN2_ERR_NULL;
    if (!d->k_heads) k = k_out = nullptr;
    const int64_t qn = dense_bytes(d, d->q_heads), kn = dense_bytes(d, d->k_heads);
    const int64_t wn = d->dim * (d->weight_dtype == GDN2_BF16 ? 2 : 4);
    // an input in whose place its output goes
    const bool q_here = q == q_out && d->q_stride == d->q_heads * d->dim, k_here = k == k_out && d->k_stride == d->k_heads * d->dim;
    const Span qi{q, strided_bytes(d, d->q_heads, d->q_stride)}, ki{k, strided_bytes(d, d->k_heads, d->k_stride)};
    const Span qo{q_out, qn}, ko{k_out, kn};
    if (!disjoint({qo, ko}, {{freq, 4 * d->rotary}, {positions, 4 * d->period}, {qw, wn}, {kw, wn}})) return GDN2_ERR_ALIAS;
    if ((!q_here && overlap(qo, qi)) || overlap(qo, ki) || (!k_here && overlap(ko, ki)) || overlap(ko, qi)) return GDN2_ERR_ALIAS;
    RotaryArgs a = args_of(d, freq, positions);
    a.part[0].x = q; a.part[0].w = qw; a.part[0].y = q_out;
    a.part[1].x = k; a.part[1].w = kw; a.part[1].y = k_out;
    a.mode = norm ? gdn2::ROTARY_NORM : gdn2::ROTARY_TURN;
    if (back) a.sin_mag = -a.sin_mag;
    return hip_status(gdn2::launch_rotary(a, nullptr, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

gdn2_status gdn2_rotary_fwd(const gdn2_rotary_desc *d, const void *q, const void *k, const double *freq,
                            const int32_t *positions, void *q_out, void *k_out, void *stream) {
    return forward(d, false, false, q, k, nullptr, nullptr, freq, positions, q_out, k_out, stream);
}

gdn2_status gdn2_rotary_bwd(const gdn2_rotary_desc *d, const void *d_q_out, const void *d_k_out, const double *freq,
                            const int32_t *positions, void *dq, void *dk, void *stream) {
    return forward(d, false, true, d_q_out, d_k_out, nullptr, nullptr, freq, positions, dq, dk, stream);
}

gdn2_status gdn2_qk_norm_fwd(const gdn2_rotary_desc *d, const void *q, const void *k, const void *q_weight,
                             const void *k_weight, const double *freq, const int32_t *positions, void *q_out, void *k_out,
                             void *stream) {
    return forward(d, true, false, q, k, q_weight, k_weight, freq, positions, q_out, k_out, stream);
}

gdn2_status gdn2_qk_norm_bwd_workspace(const gdn2_rotary_desc *d, size_t *bytes) {
    if (!bytes) return GDN2_ERR_NULL;
    const gdn2_status st = check(d, true);
    if (st != GDN2_OK) return st;
    *bytes = d->tokens ? gdn2::rotary_bwd_workspace(args_of(d, nullptr, nullptr)) : 0;
    return GDN2_OK;
}

gdn2_status gdn2_qk_norm_bwd(const gdn2_rotary_desc *d, const void *d_q_out, const void *d_k_out, const void *q, const void *k,
                             const void *q_weight, const void *k_weight, const double *freq, const int32_t *positions,
                             void *dq, void *dk, void *d_q_weight, void *d_k_weight, void *workspace, size_t ws_bytes,
                             void *stream) {
    size_t need = 0;
    const gdn2_status st = gdn2_qk_norm_bwd_workspace(d, &need);
    if (st != GDN2_OK) return st;
    const bool work = d->tokens > 0, sums = d_q_weight || d_k_weight;
    if (work && (!d_q_out || !q || !dq || (d->k_heads && (!d_k_out || !k || !dk)) || (d->rotary && !freq))) return GDN2_ERR_NULL;
    if (work && sums && (!workspace || !workspace_ok(workspace, ws_bytes, need))) return GDN2_ERR_WORKSPACE;
    if (!d->k_heads) k = d_k_out = dk = nullptr;
    const int64_t qn = dense_bytes(d, d->q_heads), kn = dense_bytes(d, d->k_heads);
    const int64_t wn = d->dim * (d->weight_dtype == GDN2_BF16 ? 2 : 4);
    if (!disjoint({{dq, qn}, {dk, kn}, {d_q_weight, wn}, {d_k_weight, wn}, {workspace, static_cast<int64_t>(ws_bytes)}},
                  {{d_q_out, qn}, {d_k_out, kn}, {q, strided_bytes(d, d->q_heads, d->q_stride)},
                   {k, strided_bytes(d, d->k_heads, d->k_stride)}, {q_weight, wn}, {k_weight, wn}, {freq, 4 * d->rotary},
                   {positions, 4 * d->period}}))
        return GDN2_ERR_ALIAS;
    hipStream_t s = static_cast<hipStream_t>(stream);
    // sums over nothing: no tokens, or a weight without heads
    hipError_t e = hipSuccess;
    if (d_q_weight && !work) e = gdn2::launch_norm_zero(d_q_weight, d->dim, d->weight_dtype == GDN2_BF16, s);
    if (d_k_weight && (!work || !d->k_heads) && e == hipSuccess)
        e = gdn2::launch_norm_zero(d_k_weight, d->dim, d->weight_dtype == GDN2_BF16, s);
    if (!work || e != hipSuccess) return hip_status(e);
    RotaryArgs a = args_of(d, freq, positions);
    a.part[0].x = q; a.part[0].dy = d_q_out; a.part[0].w = q_weight; a.part[0].y = dq; a.part[0].dw = d_q_weight;
    a.part[1].x = k; a.part[1].dy = d_k_out; a.part[1].w = k_weight; a.part[1].y = dk;
    a.part[1].dw = d->k_heads ? d_k_weight : nullptr;
    a.mode = gdn2::ROTARY_NORM_BWD;
    a.sin_mag = -a.sin_mag;
    return hip_status(gdn2::launch_rotary(a, workspace, s));
}

}  // extern "C"
