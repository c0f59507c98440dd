// linear_api.hip -- the C ABI of the linear-attention and layer-norm calls
// declared in include/gdn2.h: host-side validation, then dispatch to the
// gfx950 kernels on the caller's stream.
//
// Validation never touches the GPU, so every error path is reachable (and
// tested) on a machine without one.  No allocation, no global mutable state.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "gdn2.h"
#include "kernels.h"
#include "linear.h"

namespace {

using gdn2::LinArgs;
using gdn2::LinStepArgs;
using gdn2::NormArgs;

struct Span {
    const void *p;
    int64_t bytes;
};

bool overlap(const Span &a, const Span &b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + static_cast<uintptr_t>(b.bytes) && y < x + static_cast<uintptr_t>(a.bytes);
}

// Outputs overlap neither the inputs nor each other.
bool disjoint(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (const Span *o = outs.begin(); o != outs.end(); ++o) {
        for (const Span &i : ins)
            if (overlap(*o, i)) return false;
        for (const Span *x = o + 1; x != outs.end(); ++x)
            if (overlap(*o, *x)) return false;
    }
    return true;
}

// a*b*.. fits in int64
bool product_ok(std::initializer_list<int64_t> fs) {
    int64_t x = 1;
    for (int64_t f : fs) {
        if (f < 0) return false;
        if (f != 0 && x > INT64_MAX / f) return false;
        x *= f;
    }
    return true;
}

gdn2_status hip_status(hipError_t e) { return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP; }

bool workspace_ok(const void *ws, size_t have, size_t need) {
    return have >= need && (reinterpret_cast<uintptr_t>(ws) & 255) == 0;
}

gdn2_status check_linear(const gdn2_linear_desc *d, bool packed) {
    if (!d) return GDN2_ERR_NULL;
    if (d->batch < 0 || d->seqlen < 0 || d->heads < 1 || d->dk < 1 || d->dv < 1 || d->reserved != 0) return GDN2_ERR_SHAPE;
    if (d->dtype != GDN2_F32 && d->dtype != GDN2_BF16) return GDN2_ERR_DTYPE;
    if (d->decay_kind != GDN2_DECAY_TOKEN && d->decay_kind != GDN2_DECAY_HEAD) return GDN2_ERR_SHAPE;
    if (packed && (d->seqlen > INT32_MAX || d->batch >= INT32_MAX)) return GDN2_ERR_SHAPE;  // int32 offsets
    if (d->dk > 128 || d->dv > 128) return GDN2_ERR_UNSUPPORTED;
    const int64_t dmax = d->dk > d->dv ? d->dk : d->dv;
    if (!product_ok({packed ? 1 : d->batch, d->seqlen, d->heads, dmax, 16}) ||
        !product_ok({d->batch, d->heads, d->dk, d->dv, 16}))
        return GDN2_ERR_SHAPE;
    // 32-bit offsets inside a chunk, 2^32 lanes a launch over the chains
    if (d->seqlen > INT32_MAX || d->heads > 65535 || d->batch * d->heads >= (INT64_C(1) << 20)) return GDN2_ERR_UNSUPPORTED;
    return GDN2_OK;
}

struct Bytes {
    int64_t qk, v, la, st;
};

Bytes bytes_of(const gdn2_linear_desc *d, bool packed) {
    Bytes b;
    const int64_t esz = d->dtype == GDN2_BF16 ? 2 : 4, tok = (packed ? 1 : d->batch) * d->seqlen * d->heads;
    b.qk = tok * d->dk * esz;
    b.v = tok * d->dv * esz;
    b.la = 4 * (d->decay_kind == GDN2_DECAY_TOKEN ? tok : d->heads);
    b.st = d->batch * d->heads * d->dk * d->dv * 4;
    return b;
}

LinArgs args_of(const gdn2_linear_desc *d, const int32_t *cu, const void *q, const void *k, const void *v, const float *la,
                const float *s0) {
    LinArgs a = {};
    a.q = q; a.k = k; a.v = v; a.la = la; a.s0 = s0; a.cu = cu;
    a.N = d->batch; a.T = d->seqlen; a.H = d->heads; a.dk = d->dk; a.dv = d->dv;
    a.bf16 = d->dtype == GDN2_BF16;
    a.la_tok = d->decay_kind == GDN2_DECAY_TOKEN;
    a.scale = d->q_scale;
    return a;
}

// stands for the offsets of a packed request where only its sizes matter
const int32_t packed_mark = 0;

gdn2_status space_of(const gdn2_linear_desc *d, bool packed, bool backward, size_t *bytes) {
    if (!bytes) return GDN2_ERR_NULL;
    const gdn2_status st = check_linear(d, packed);
    if (st != GDN2_OK) return st;
    const LinArgs a = args_of(d, packed ? &packed_mark : nullptr, nullptr, nullptr, nullptr, nullptr, nullptr);
    if (!gdn2::linear_fits(a, backward)) return GDN2_ERR_UNSUPPORTED;
    *bytes = backward ? gdn2::linear_bwd_workspace(a) : gdn2::linear_fwd_workspace(a);
    return GDN2_OK;
}

gdn2_status forward(const gdn2_linear_desc *d, bool packed, const int32_t *cu, const void *q, const void *k, const void *v,
                    const float *la, const float *s0, void *o, float *s_out, void *ws, size_t ws_bytes, void *stream) {
    size_t need = 0;
    const gdn2_status st = space_of(d, packed, false, &need);
    if (st != GDN2_OK) return st;
    const bool use_ws = ws != nullptr && ws_bytes > 0;
    if (use_ws && !workspace_ok(ws, ws_bytes, need)) return GDN2_ERR_WORKSPACE;
    const bool work = d->batch > 0 && d->seqlen > 0;
    if (packed && d->batch > 0 && !cu) return GDN2_ERR_NULL;
    if (work && (!q || !k || !v || !la || !o)) return GDN2_ERR_NULL;
    const Bytes b = bytes_of(d, packed);
    const Span so{s_out, b.st}, si{s0, b.st}, wsp{use_ws ? ws : nullptr, static_cast<int64_t>(ws_bytes)};
    const Span offs{cu, packed ? 4 * (d->batch + 1) : 0};
    if (!disjoint({{o, b.v}, so, wsp}, {{q, b.qk}, {k, b.qk}, {v, b.v}, {la, b.la}, offs})) return GDN2_ERR_ALIAS;
    if (!disjoint({{o, b.v}, wsp}, {si})) return GDN2_ERR_ALIAS;
    if (s0 != s_out && overlap(si, so)) return GDN2_ERR_ALIAS;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (d->batch == 0) return GDN2_OK;
    if (!work) {
        if (s_out && s_out != s0) return hip_status(gdn2::launch_state_copy(s0, s_out, b.st / 4, s));
        return GDN2_OK;
    }
    LinArgs a = args_of(d, packed ? cu : nullptr, q, k, v, la, s0);
    a.o = o;
    a.s_out = s_out;
    return hip_status(gdn2::launch_linear_fwd(a, use_ws && need > 0 ? ws : nullptr, s));
}

gdn2_status backward(const gdn2_linear_desc *d, bool packed, const int32_t *cu, const void *q, const void *k, const void *v,
                     const float *la, const float *s0, const void *d_o, const float *d_sT, void *dq, void *dk, void *dv,
                     float *d_la, float *d_s0, void *ws, size_t ws_bytes, void *stream) {
    size_t need = 0;
    const gdn2_status st = space_of(d, packed, true, &need);
    if (st != GDN2_OK) return st;
    const bool work = d->batch > 0 && d->seqlen > 0;
    if (packed && d->batch > 0 && !cu) return GDN2_ERR_NULL;
    if (work && (!q || !k || !v || !la || !d_o || !dq || !dk || !dv || !d_la)) return GDN2_ERR_NULL;
    const bool per_head = d->decay_kind == GDN2_DECAY_HEAD;
    if (per_head && !d_la) return GDN2_ERR_NULL;
    if (work && (!ws || !workspace_ok(ws, ws_bytes, need))) return GDN2_ERR_WORKSPACE;
    const Bytes b = bytes_of(d, packed);
    const Span offs{cu, packed ? 4 * (d->batch + 1) : 0}, wsp{ws, static_cast<int64_t>(ws_bytes)};
    if (!disjoint({{dq, b.qk}, {dk, b.qk}, {dv, b.v}, {d_la, b.la}, {d_s0, b.st}, wsp},
                  {{q, b.qk}, {k, b.qk}, {v, b.v}, {la, b.la}, {s0, b.st}, {d_o, b.v}, {d_sT, b.st}, offs}))
        return GDN2_ERR_ALIAS;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (!work) {  // no token: the state's gradient passes through
        hipError_t e = hipSuccess;
        if (per_head) e = gdn2::launch_state_copy(nullptr, d_la, d->heads, s);
        if (e == hipSuccess && d_s0) e = gdn2::launch_state_copy(d_sT, d_s0, b.st / 4, s);
        return hip_status(e);
    }
    LinArgs a = args_of(d, packed ? cu : nullptr, q, k, v, la, s0);
    a.d_o = d_o; a.d_sT = d_sT; a.dq = dq; a.dk_out = dk; a.dv_out = dv; a.d_la = d_la; a.d_s0 = d_s0;
    return hip_status(gdn2::launch_linear_bwd(a, ws, s));
}

gdn2_status check_norm(const gdn2_norm_desc *d) {
    if (!d) return GDN2_ERR_NULL;
    if (d->rows < 0 || d->groups < 1 || d->dim < 1 || d->rows % d->groups != 0 || d->reserved != 0) return GDN2_ERR_SHAPE;
    if ((d->dtype != GDN2_F32 && d->dtype != GDN2_BF16) || (d->weight_dtype != GDN2_F32 && d->weight_dtype != GDN2_BF16))
        return GDN2_ERR_DTYPE;
    if (!(d->eps >= 0.f)) return GDN2_ERR_SHAPE;
    if (!product_ok({d->rows, d->dim, 16})) return GDN2_ERR_SHAPE;
    // 2^32 lanes a launch: 1024 for 16 columns of a weight row
    if (d->dim > 16384 || d->rows > INT32_MAX || d->groups >= (INT64_C(1) << 22) / ((d->dim + 15) / 16))
        return GDN2_ERR_UNSUPPORTED;
    return GDN2_OK;
}

NormArgs norm_args(const gdn2_norm_desc *d) {
    NormArgs a = {};
    a.rows = d->rows; a.G = d->groups; a.D = d->dim;
    a.bf16 = d->dtype == GDN2_BF16;
    a.w_bf16 = d->weight_dtype == GDN2_BF16;
    a.eps = d->eps;
    return a;
}

}  // namespace

extern "C" {

gdn2_status gdn2_linear_fwd_workspace(const gdn2_linear_desc *d, size_t *bytes) { return space_of(d, false, false, bytes); }
gdn2_status gdn2_linear_fwd_varlen_workspace(const gdn2_linear_desc *d, size_t *bytes) { return space_of(d, true, false, bytes); }
gdn2_status gdn2_linear_bwd_workspace(const gdn2_linear_desc *d, size_t *bytes) { return space_of(d, false, true, bytes); }
gdn2_status gdn2_linear_bwd_varlen_workspace(const gdn2_linear_desc *d, size_t *bytes) { return space_of(d, true, true, bytes); }

gdn2_status gdn2_linear_fwd(const gdn2_linear_desc *d, const void *q, const void *k, const void *v, const float *log_decay,
                            const float *state0, void *o, float *state_out, void *workspace, size_t ws_bytes, void *stream) {
    return forward(d, false, nullptr, q, k, v, log_decay, state0, o, state_out, workspace, ws_bytes, stream);
}

gdn2_status gdn2_linear_fwd_varlen(const gdn2_linear_desc *d, const int32_t *cu_seqlens, const void *q, const void *k,
                                   const void *v, const float *log_decay, const float *state0, void *o, float *state_out,
                                   void *workspace, size_t ws_bytes, void *stream) {
    return forward(d, true, cu_seqlens, q, k, v, log_decay, state0, o, state_out, workspace, ws_bytes, stream);
}

gdn2_status gdn2_linear_bwd(const gdn2_linear_desc *d, const void *q, const void *k, const void *v, const float *log_decay,
                            const float *state0, const void *d_o, const float *d_state_out, void *dq, void *dk, void *dv,
                            float *d_log_decay, float *d_state0, void *workspace, size_t ws_bytes, void *stream) {
    return backward(d, false, nullptr, q, k, v, log_decay, state0, d_o, d_state_out, dq, dk, dv, d_log_decay, d_state0,
                    workspace, ws_bytes, stream);
}

gdn2_status gdn2_linear_bwd_varlen(const gdn2_linear_desc *d, const int32_t *cu_seqlens, const void *q, const void *k,
                                   const void *v, const float *log_decay, const float *state0, const void *d_o,
                                   const float *d_state_out, void *dq, void *dk, void *dv, float *d_log_decay,
                                   float *d_state0, void *workspace, size_t ws_bytes, void *stream) {
    return backward(d, true, cu_seqlens, q, k, v, log_decay, state0, d_o, d_state_out, dq, dk, dv, d_log_decay, d_state0,
                    workspace, ws_bytes, stream);
}

gdn2_status gdn2_linear_step(const gdn2_linear_desc *d, const void *q, const void *k, const void *v, const float *log_decay,
                             float *state, void *o, void *stream) {
    const gdn2_status st = check_linear(d, false);
    if (st != GDN2_OK) return st;
    if (d->seqlen != 1) return GDN2_ERR_SHAPE;
    if (d->batch == 0) return GDN2_OK;
    if (!q || !k || !v || !log_decay || !state || !o) return GDN2_ERR_NULL;
    const Bytes b = bytes_of(d, false);
    if (!disjoint({{o, b.v}, {state, b.st}}, {{q, b.qk}, {k, b.qk}, {v, b.v}, {log_decay, b.la}})) return GDN2_ERR_ALIAS;
    LinStepArgs a = {};
    a.q = q; a.k = k; a.v = v; a.la = log_decay; a.state = state; a.o = o;
    a.N = d->batch; a.H = d->heads; a.dk = d->dk; a.dv = d->dv;
    a.bf16 = d->dtype == GDN2_BF16;
    a.la_tok = d->decay_kind == GDN2_DECAY_TOKEN;
    a.scale = d->q_scale;
    return hip_status(gdn2::launch_linear_step(a, static_cast<hipStream_t>(stream)));
}

gdn2_status gdn2_layer_norm_fwd(const gdn2_norm_desc *d, const void *x, const void *weight, const void *bias, void *y,
                                float *mean, float *rstd, void *stream) {
    const gdn2_status st = check_norm(d);
    if (st != GDN2_OK) return st;
    if (d->rows == 0) return GDN2_OK;
    if (!x || !y) return GDN2_ERR_NULL;
    const int64_t n = d->rows * d->dim * (d->dtype == GDN2_BF16 ? 2 : 4);
    const int64_t w = d->groups * d->dim * (d->weight_dtype == GDN2_BF16 ? 2 : 4);
    if (!disjoint({{y, n}, {mean, 4 * d->rows}, {rstd, 4 * d->rows}}, {{x, n}, {weight, w}, {bias, w}})) return GDN2_ERR_ALIAS;
    NormArgs a = norm_args(d);
    a.x = x; a.w = weight; a.b = bias; a.y = y; a.mean = mean; a.rstd = rstd;
    return hip_status(gdn2::launch_norm_fwd(a, static_cast<hipStream_t>(stream)));
}

gdn2_status gdn2_layer_norm_bwd_workspace(const gdn2_norm_desc *d, size_t *bytes) {
    if (!bytes) return GDN2_ERR_NULL;
    const gdn2_status st = check_norm(d);
    if (st != GDN2_OK) return st;
    *bytes = d->rows ? gdn2::norm_bwd_workspace(norm_args(d)) : 0;
    return GDN2_OK;
}

gdn2_status gdn2_layer_norm_bwd(const gdn2_norm_desc *d, const void *dy, const void *x, const void *weight, const float *mean,
                                const float *rstd, void *dx, void *d_weight, void *d_bias, void *workspace, size_t ws_bytes,
                                void *stream) {
    size_t need = 0;
    const gdn2_status st = gdn2_layer_norm_bwd_workspace(d, &need);
    if (st != GDN2_OK) return st;
    if (d->rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return GDN2_ERR_NULL;
    const bool sums = d_weight || d_bias;
    if (d->rows > 0 && sums && (!workspace || !workspace_ok(workspace, ws_bytes, need))) return GDN2_ERR_WORKSPACE;
    const int64_t n = d->rows * d->dim * (d->dtype == GDN2_BF16 ? 2 : 4);
    const int64_t wn = d->groups * d->dim, w = wn * (d->weight_dtype == GDN2_BF16 ? 2 : 4);
    if (!disjoint({{dx, n}, {d_weight, w}, {d_bias, w}, {workspace, static_cast<int64_t>(ws_bytes)}},
                  {{dy, n}, {x, n}, {weight, w}, {mean, 4 * d->rows}, {rstd, 4 * d->rows}}))
        return GDN2_ERR_ALIAS;
    hipStream_t s = static_cast<hipStream_t>(stream);
    NormArgs a = norm_args(d);
    a.dy = dy; a.x = x; a.w = weight; a.dx = dx; a.dw = d_weight; a.db = d_bias;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    if (d->rows == 0) {  // sums over no row
        hipError_t e = hipSuccess;
        for (void *p : {d_weight, d_bias})
            if (p && e == hipSuccess) e = gdn2::launch_norm_zero(p, wn, a.w_bf16, s);
        return hip_status(e);
    }
    return hip_status(gdn2::launch_norm_bwd(a, workspace, s));
}

}  // extern "C"
