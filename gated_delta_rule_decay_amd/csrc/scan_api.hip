// scan_api.hip -- the C ABI of the gated scan declared in include/gdn2.h:
// host-side validation, then dispatch to the gfx950 kernels on the caller's
// stream.  Validation never touches the GPU.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "api_check.h"
#include "gdn2.h"
#include "kernels.h"
#include "scan.h"

namespace {

using namespace gdn2::api;
using gdn2::ScanArgs;

// stands for the offsets of a packed request where only its sizes matter
const int32_t packed_mark = 0;

ScanArgs args_of(const gdn2_scan_desc *d, const int32_t *cu, const void *x, const void *gate, const float *s0) {
    ScanArgs a = {};
    a.x = x; a.gate = gate; a.s0 = s0; a.cu = cu;
    a.N = d->batch; a.T = d->seqlen; a.D = d->dim;
    a.bf16 = d->dtype == GDN2_BF16;
    a.gate_bf16 = d->gate_dtype == GDN2_BF16;
    a.logits = d->gate_logits != 0;
    a.comp = d->complement != 0;
    return a;
}

gdn2_status check(const gdn2_scan_desc *d, bool packed) {
    if (!d) return GDN2_ERR_NULL;
    if (d->batch < 0 || d->seqlen < 0 || d->dim < 1) return GDN2_ERR_SHAPE;
    if ((d->dtype != GDN2_F32 && d->dtype != GDN2_BF16) || (d->gate_dtype != GDN2_F32 && d->gate_dtype != GDN2_BF16))
        return GDN2_ERR_DTYPE;
    if (packed && (d->seqlen > INT32_MAX || d->batch >= INT32_MAX)) return GDN2_ERR_SHAPE;  // int32 offsets
    if (!product_ok({packed ? 1 : d->batch, d->seqlen, d->dim, 16}) || !product_ok({d->batch, d->dim, 16})) return GDN2_ERR_SHAPE;
    if (d->seqlen > INT32_MAX || d->batch > INT32_MAX || d->dim > INT32_MAX) return GDN2_ERR_UNSUPPORTED;
    if (!gdn2::scan_fits(args_of(d, packed ? &packed_mark : nullptr, nullptr, nullptr, nullptr))) return GDN2_ERR_UNSUPPORTED;
    return GDN2_OK;
}

struct Bytes {
    int64_t x, gate, state, marks, offs;
};

Bytes bytes_of(const gdn2_scan_desc *d, bool packed) {
    Bytes b;
    const int64_t rows = packed ? 1 : d->batch, n = rows * d->seqlen * d->dim;
    b.x = n * (d->dtype == GDN2_BF16 ? 2 : 4);
    b.gate = n * (d->gate_dtype == GDN2_BF16 ? 2 : 4);
    b.state = d->batch * d->dim * 4;
    b.marks = rows * ((d->seqlen + gdn2::SCAN_MARK - 1) / gdn2::SCAN_MARK) * d->dim * 4;
    b.offs = packed ? 4 * (d->batch + 1) : 0;
    return b;
}

gdn2_status space_of(const gdn2_scan_desc *d, bool packed, size_t *bytes) {
    if (!bytes) return GDN2_ERR_NULL;
    const gdn2_status st = check(d, packed);
    if (st != GDN2_OK) return st;
    *bytes = gdn2::scan_workspace(args_of(d, packed ? &packed_mark : nullptr, nullptr, nullptr, nullptr));
    return GDN2_OK;
}

gdn2_status forward(const gdn2_scan_desc *d, bool packed, const int32_t *cu, const void *x, const void *gate, const float *s0,
                    void *y, float *s_out, float *marks, void *ws, size_t ws_bytes, void *stream) {
    size_t need = 0;
    const gdn2_status st = space_of(d, packed, &need);
    if (st != GDN2_OK) return st;
    const bool work = d->batch > 0 && d->seqlen > 0;
    if (packed && d->batch > 0 && !cu) return GDN2_ERR_NULL;
    if (work && (!x || !gate || !y)) return GDN2_ERR_NULL;
    if (work && need && (!ws || !workspace_ok(ws, ws_bytes, need))) return GDN2_ERR_WORKSPACE;
    const Bytes b = bytes_of(d, packed);
    const Span so{s_out, b.state}, si{s0, b.state}, yo{y, b.x}, mo{marks, b.marks}, wsp{ws, static_cast<int64_t>(ws_bytes)};
    if (!disjoint({yo, so, mo, wsp}, {{x, b.x}, {gate, b.gate}, {cu, b.offs}})) return GDN2_ERR_ALIAS;
    if (!disjoint({yo, mo, wsp}, {si})) return GDN2_ERR_ALIAS;
    if (s0 != s_out && overlap(si, so)) return GDN2_ERR_ALIAS;
    if (d->batch == 0) return GDN2_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (!work) {
        if (s_out && s_out != s0) return hip_status(gdn2::launch_state_copy(s0, s_out, b.state / 4, s));
        return GDN2_OK;
    }
    ScanArgs a = args_of(d, packed ? cu : nullptr, x, gate, s0);
    a.y = y; a.s_out = s_out; a.marks = marks;
    return hip_status(gdn2::launch_scan_fwd(a, ws, s));
}

gdn2_status backward(const gdn2_scan_desc *d, bool packed, const int32_t *cu, const void *dy, const void *x, const void *gate,
                     const float *marks, const float *s0, const float *d_sT, void *dx, void *d_gate, float *d_s0, void *ws,
                     size_t ws_bytes, void *stream) {
    size_t need = 0;
    const gdn2_status st = space_of(d, packed, &need);
    if (st != GDN2_OK) return st;
    const bool work = d->batch > 0 && d->seqlen > 0;
    if (packed && d->batch > 0 && !cu) return GDN2_ERR_NULL;
    if (work && (!dy || !x || !gate || !marks || !dx || !d_gate)) return GDN2_ERR_NULL;
    if (work && need && (!ws || !workspace_ok(ws, ws_bytes, need))) return GDN2_ERR_WORKSPACE;
    const Bytes b = bytes_of(d, packed);
    if (!disjoint({{dx, b.x}, {d_gate, b.gate}, {d_s0, b.state}, {ws, static_cast<int64_t>(ws_bytes)}},
                  {{dy, b.x}, {x, b.x}, {gate, b.gate}, {marks, b.marks}, {s0, b.state}, {d_sT, b.state}, {cu, b.offs}}))
        return GDN2_ERR_ALIAS;
    if (d->batch == 0) return GDN2_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (!work) {  // no token: the state's gradient passes through
        if (d_s0) return hip_status(gdn2::launch_state_copy(d_sT, d_s0, b.state / 4, s));
        return GDN2_OK;
    }
    ScanArgs a = args_of(d, packed ? cu : nullptr, x, gate, s0);
    a.marks = const_cast<float *>(marks);
    a.dy = dy; a.d_sT = d_sT; a.dx = dx; a.d_gate = d_gate; a.d_s0 = d_s0;
    return hip_status(gdn2::launch_scan_bwd(a, ws, s));
}

}  // namespace

extern "C" {

gdn2_status gdn2_scan_fwd_workspace(const gdn2_scan_desc *d, size_t *bytes) { return space_of(d, false, bytes); }
gdn2_status gdn2_scan_fwd_varlen_workspace(const gdn2_scan_desc *d, size_t *bytes) { return space_of(d, true, bytes); }
gdn2_status gdn2_scan_bwd_workspace(const gdn2_scan_desc *d, size_t *bytes) { return space_of(d, false, bytes); }
gdn2_status gdn2_scan_bwd_varlen_workspace(const gdn2_scan_desc *d, size_t *bytes) { return space_of(d, true, bytes); }

gdn2_status gdn2_scan_fwd(const gdn2_scan_desc *d, const void *x, const void *log_decay, const float *state0, void *y,
                          float *state_out, float *marks, void *workspace, size_t ws_bytes, void *stream) {
    return forward(d, false, nullptr, x, log_decay, state0, y, state_out, marks, workspace, ws_bytes, stream);
}

gdn2_status gdn2_scan_fwd_varlen(const gdn2_scan_desc *d, const int32_t *cu_seqlens, const void *x, const void *log_decay,
                                 const float *state0, void *y, float *state_out, float *marks, void *workspace,
                                 size_t ws_bytes, void *stream) {
    return forward(d, true, cu_seqlens, x, log_decay, state0, y, state_out, marks, workspace, ws_bytes, stream);
}

gdn2_status gdn2_scan_bwd(const gdn2_scan_desc *d, const void *dy, const void *x, const void *log_decay, const float *marks,
                          const float *state0, const float *d_state_out, void *dx, void *d_log_decay, float *d_state0,
                          void *workspace, size_t ws_bytes, void *stream) {
    return backward(d, false, nullptr, dy, x, log_decay, marks, state0, d_state_out, dx, d_log_decay, d_state0, workspace,
                    ws_bytes, stream);
}

gdn2_status gdn2_scan_bwd_varlen(const gdn2_scan_desc *d, const int32_t *cu_seqlens, const void *dy, const void *x,
                                 const void *log_decay, const float *marks, const float *state0, const float *d_state_out,
                                 void *dx, void *d_log_decay, float *d_state0, void *workspace, size_t ws_bytes, void *stream) {
    return backward(d, true, cu_seqlens, dy, x, log_decay, marks, state0, d_state_out, dx, d_log_decay, d_state0, workspace,
                    ws_bytes, stream);
}

gdn2_status gdn2_scan_step(const gdn2_scan_desc *d, const void *x, const void *log_decay, float *state, void *y, void *stream) {
    const gdn2_status st = check(d, false);
    if (st != GDN2_OK) return st;
    if (d->seqlen != 1) return GDN2_ERR_SHAPE;
    if (d->batch == 0) return GDN2_OK;
    if (!x || !log_decay || !state || !y) return GDN2_ERR_NULL;
    const Bytes b = bytes_of(d, false);
    if (!disjoint({{y, b.x}, {state, b.state}}, {{x, b.x}, {log_decay, b.gate}})) return GDN2_ERR_ALIAS;
    gdn2::ScanStepArgs a = {};
    a.x = x; a.gate = log_decay; a.state = state; a.y = y;
    a.n = d->batch * d->dim;
    a.bf16 = d->dtype == GDN2_BF16;
    a.gate_bf16 = d->gate_dtype == GDN2_BF16;
    a.logits = d->gate_logits != 0;
    a.comp = d->complement != 0;
    return hip_status(gdn2::launch_scan_step(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
