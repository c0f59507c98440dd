// linear.h -- internal interface of the linear-attention and layer-norm
// kernels (linear_chunk.hip, linear_step.hip, layer_norm.hip) to the C-ABI
// layer (linear_api.hip).  Not installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn2 {

// A chunked linear-attention request.  Sequences: N of T tokens each
// ([N,T,H,d]), or with `cu` N packed along one axis of T tokens.
struct LinArgs {
    const void *q, *k, *v;  // bf16 or fp32
    const float *la;        // [.., T, H] (la_tok) or [H]
    const float *s0;        // [N,H,dk,dv] or nullptr (zeros)
    void *o;                // like v, or nullptr (backward)
    float *s_out;           // [N,H,dk,dv] or nullptr
    const int32_t *cu;      // device [N+1] or nullptr
    int64_t N, T, H, dk, dv;
    int bf16, la_tok;
    float scale;
    // backward
    const void *d_o;        // like v
    const float *d_sT;      // [N,H,dk,dv] or nullptr
    void *dq, *dk_out, *dv_out;
    float *d_la;            // like la
    float *d_s0;            // [N,H,dk,dv] or nullptr
};

// whether every launch of a request stays below 2^32 lanes
bool linear_fits(const LinArgs &a, bool backward);
size_t linear_fwd_workspace(const LinArgs &a);
size_t linear_bwd_workspace(const LinArgs &a);
hipError_t launch_linear_fwd(const LinArgs &a, void *ws, hipStream_t s);  // ws nullptr: one pass
hipError_t launch_linear_bwd(const LinArgs &a, void *ws, hipStream_t s);

struct LinStepArgs {
    const void *q, *k, *v;  // [N,H,dk] / [N,H,dv]
    const float *la;        // [N,H] (la_tok) or [H]
    float *state;           // [N,H,dk,dv], in place
    void *o;                // [N,H,dv]
    int64_t N, H, dk, dv;
    int bf16, la_tok;
    float scale;
};
hipError_t launch_linear_step(const LinStepArgs &a, hipStream_t s);

struct NormArgs {
    const void *x;          // [rows, D], bf16 or fp32
    const void *w, *b;      // [G, D]; nullptr: ones / zeros
    void *y;                // [rows, D] (forward)
    float *mean, *rstd;     // [rows]
    const void *dy;         // [rows, D] (backward)
    void *dx;
    void *dw, *db;          // [G, D] or nullptr
    int64_t rows, G, D;     // row r uses weight row r % G
    int bf16, w_bf16;
    float eps;
};
size_t norm_bwd_workspace(const NormArgs &a);
hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t s);
hipError_t launch_norm_zero(void *p, int64_t n, int bf16, hipStream_t s);  // n zeros
hipError_t launch_norm_bwd(const NormArgs &a, void *ws, hipStream_t s);

}  // namespace gdn2
