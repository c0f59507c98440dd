// rotary.h -- internal interface of the rotary and query/key norm kernels
// (rotary.hip) to the C-ABI layer (rotary_api.hip).  Not installed, not part
// of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn2 {

// q or k of a request.
struct RotaryPart {
    const void *x;   // [tokens, H, d], `stride` elements from token to token
    const void *dy;  // norm backward: the gradient of the output, contiguous
    const void *w;   // [d] or nullptr (ones)
    void *y;         // contiguous: the output, or x's gradient
    void *dw;        // [d] or nullptr
    int64_t stride;
    int H;           // 0: nothing to do
};

enum RotaryMode { ROTARY_TURN = 0, ROTARY_NORM = 1, ROTARY_NORM_BWD = 2 };

struct RotaryArgs {
    RotaryPart part[2];  // q, k
    const double *freq;  // [rot/2]
    const int32_t *pos;  // [period] or nullptr
    int64_t offset;
    int tokens, period, d, rot;
    int mode;            // RotaryMode
    int bf16, w_bf16, inter, l2;
    float eps, cos_mag, sin_mag;  // factors of cos and sin (backward: sin negative)
};

size_t rotary_bwd_workspace(const RotaryArgs &a);
hipError_t launch_rotary(const RotaryArgs &a, void *ws, hipStream_t s);

}  // namespace gdn2
