// linear_step.hip -- one decode step of linear attention per (sequence,
// head), the state in place:  S <- e^{la} S + k v^T,  o = scale S^T q.
//
// Bound by HBM: the state is read and written once (8 dk dv bytes against
// 4 dk dv operations).  The columns of the state are independent of each
// other, so a workgroup takes a slab of CW columns of one head: 128 where
// there are heads enough to fill the chip, 32 where there are few and the
// latency of one workgroup's loads counts.  All of a lane's loads are issued
// before the first is used.
#include "common.h"
#include "linear.h"

namespace gdn2 {
namespace {

template <int V>
struct Vec {
    float e[V];
};

template <int V, int CW>
__global__ void __launch_bounds__(256) linear_step_kernel(LinStepArgs a, int slabs) {
    constexpr int CL = CW / V, RG = 256 / CL, ROWS = (128 + RG - 1) / RG;  // lanes of a row, row groups
    __shared__ float s_k[128], s_q[128];
    __shared__ float s_o[4][CW];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t head = blockIdx.x / slabs;
    const int dk = static_cast<int>(a.dk), dv = static_cast<int>(a.dv);
    const int c = static_cast<int>(blockIdx.x % slabs) * CW + (tid % CL) * V, rg = tid / CL;
    float *st = a.state + head * dk * dv;
    const bool col = c < dv;

    Vec<V> S[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int r = rg + RG * i;
        if (col && r < dk) S[i] = *reinterpret_cast<const Vec<V> *>(st + r * dv + c);
    }
    const float ea = __expf(a.la[a.la_tok ? head : head % a.H]);
    for (int i = tid; i < dk; i += 256) {
        s_k[i] = load_qkv(a.k, head * dk + i, a.bf16);
        s_q[i] = a.scale * load_qkv(a.q, head * dk + i, a.bf16);
    }
    Vec<V> v, o;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        v.e[e] = col ? load_qkv(a.v, head * dv + c + e, a.bf16) : 0.f;
        o.e[e] = 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int r = rg + RG * i;
        if (col && r < dk) {
            const float kr = s_k[r], qr = s_q[r];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                S[i].e[e] = ea * S[i].e[e] + kr * v.e[e];
                o.e[e] += qr * S[i].e[e];
            }
            *reinterpret_cast<Vec<V> *>(st + r * dv + c) = S[i];
        }
    }
#pragma unroll
    for (int m = CL; m < 64; m <<= 1)
#pragma unroll
        for (int e = 0; e < V; ++e) o.e[e] += __shfl_xor(o.e[e], m);
    if (lane < CL)
#pragma unroll
        for (int e = 0; e < V; ++e) s_o[wave][lane * V + e] = o.e[e];
    __syncthreads();
    const int oc = static_cast<int>(blockIdx.x % slabs) * CW + tid;
    if (tid < CW && oc < dv)
        store_out(static_cast<float *>(a.o), head * dv + oc, s_o[0][tid] + s_o[1][tid] + s_o[2][tid] + s_o[3][tid],
                  a.bf16);
}

template <int V, int CW>
hipError_t go(const LinStepArgs &a, hipStream_t s) {
    const int64_t slabs = (a.dv + CW - 1) / CW, grid = a.N * a.H * slabs;
    if (grid > 0x7fffffffLL) return hipErrorInvalidValue;
    hipLaunchKernelGGL((linear_step_kernel<V, CW>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, a,
                       static_cast<int>(slabs));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_step(const LinStepArgs &a, hipStream_t s) {
    const bool vec = a.dv % 4 == 0 && (reinterpret_cast<uintptr_t>(a.state) & 15) == 0;
    if (!vec) return go<1, 32>(a, s);
    return a.N * a.H >= 1024 ? go<4, 128>(a, s) : go<4, 32>(a, s);
}

}  // namespace gdn2
