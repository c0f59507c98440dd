// scan.h -- internal interface of the gated scan kernels (scan.hip) to the
// C-ABI layer (scan_api.hip).  Not installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn2 {

constexpr int SCAN_MARK = 128;  // tokens from mark to mark

struct ScanArgs {
    const void *x, *gate;    // [N,T,D], or with `cu` [T,D]
    const float *s0;         // [N,D] or nullptr (zeros)
    void *y;                 // like x (forward)
    float *s_out;            // [N,D] or nullptr
    float *marks;            // [N,ceil(T/SCAN_MARK),D]; forward: or nullptr
    const int32_t *cu;       // device [N+1] or nullptr
    int64_t N, T, D;
    int bf16, gate_bf16, logits, comp;
    // backward
    const void *dy;          // like x
    const float *d_sT;       // [N,D] or nullptr
    void *dx, *d_gate;       // like x, like gate
    float *d_s0;             // [N,D] or nullptr
};

bool scan_fits(const ScanArgs &a);  // whether the launches of a request stay in range
size_t scan_workspace(const ScanArgs &a);
hipError_t launch_scan_fwd(const ScanArgs &a, void *ws, hipStream_t s);
hipError_t launch_scan_bwd(const ScanArgs &a, void *ws, hipStream_t s);

struct ScanStepArgs {
    const void *x, *gate;  // [N,D]
    float *state;          // [N,D], in place
    void *y;
    int64_t n;             // N * D
    int bf16, gate_bf16, logits, comp;
};
hipError_t launch_scan_step(const ScanStepArgs &a, hipStream_t s);

}  // namespace gdn2
