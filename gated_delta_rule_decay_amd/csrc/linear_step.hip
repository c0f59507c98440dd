// linear_step.hip -- one decode step of linear attention per (sequence,
// head), the state in place:  S <- e^{la} S + k v^T,  o = scale S^T q.
//
// Bound by HBM: the state is read and written once (8 dk dv bytes against
// 4 dk dv operations).  The columns of the state are independent of each
// other, so a workgroup takes a slab of CW = 32 columns of one head: with few
// heads the latency of one workgroup's loads counts (16 heads of 128 x 128:
// 3.9 us, with slabs of 128 6.4), with many the slabs' loads and stores
// overlap (4096 heads: 104 us, 5.2 TB/s, 128: 114; only states that the cache
// holds gain from wide slabs, 1024 heads: 24.9 and 21.6).  All of a lane's
// loads are issued before the first is used.
#include "common.h"
#include "linear.h"

namespace gdn2 {
namespace {

constexpr int CW = 32;  // columns of a workgroup

template <int V>
struct Vec {
    float e[V];
};

template <int V>
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

template <int V>
hipError_t go(const LinStepArgs &a, hipStream_t s) {
    const int64_t slabs = (a.dv + CW - 1) / CW, grid = a.N * a.H * slabs;
    if (grid > 0x7fffffffLL) return hipErrorInvalidValue;
    hipLaunchKernelGGL((linear_step_kernel<V>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, a,
                       static_cast<int>(slabs));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_step(const LinStepArgs &a, hipStream_t s) {
    const bool vec = a.dv % 4 == 0 && (reinterpret_cast<uintptr_t>(a.state) & 15) == 0;
    return vec ? go<4>(a, s) : go<1>(a, s);
}

}  // namespace gdn2
