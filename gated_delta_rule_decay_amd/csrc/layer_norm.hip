// layer_norm.hip -- layer norm over the last axis, forward and backward.
//
//   xh = (x - mean) rstd,  y = xh w + b,  rstd = 1 / sqrt(var + eps)
//   dx = rstd (wdy - mean(wdy) - xh mean(wdy xh)),  wdy = w dy
//   dw = sum_rows dy xh,  db = sum_rows dy
//
// Bound by HBM.  A row is read once and held in registers: by 4 to 64 lanes
// of a wave (several rows a wave), or by a whole workgroup for long rows.  The
// variance is the mean square of x - mean, taken from the registers, so it
// does not cancel where the mean is large.  All sums are fp32 (the weight's
// across workgroups fp64).
#include <initializer_list>
#include <type_traits>

#include "common.h"
#include "linear.h"

namespace gdn2 {
namespace {

template <class T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<uint16_t>(uint16_t x) { return bf16_to_f32(x); }

template <class T, int VE>
struct alignas(VE * sizeof(T)) Pack {
    T e[VE];
};

// VE elements at p + c; columns past D read as zero (VE > 1: D is a multiple).
template <class T, int VE>
__device__ __forceinline__ void load_pack(const T *p, int c, int D, float (&v)[VE]) {
    Pack<T, VE> t = {};
    if (c < D) t = *reinterpret_cast<const Pack<T, VE> *>(p + c);
#pragma unroll
    for (int e = 0; e < VE; ++e) v[e] = to_f32<T>(t.e[e]);
}
template <class T, int VE>
__device__ __forceinline__ void store_pack(T *p, int c, int D, const float (&v)[VE]) {
    if (c >= D) return;
    Pack<T, VE> t;
#pragma unroll
    for (int e = 0; e < VE; ++e) {
        if constexpr (sizeof(T) == 2) t.e[e] = f32_to_bf16(v[e]);
        else t.e[e] = v[e];
    }
    *reinterpret_cast<Pack<T, VE> *>(p + c) = t;
}
// the weight's elements (bf16 or fp32), `none` without one
template <int VE>
__device__ __forceinline__ void load_weight(const void *w, int w_bf16, int64_t row, int c, int D, float none, float (&v)[VE]) {
#pragma unroll
    for (int e = 0; e < VE; ++e) v[e] = w && c + e < D ? load_qkv(w, row * D + c + e, w_bf16) : none;
}

// Sum over the lanes of a row: tpr neighbouring lanes of a wave, or (BLOCK,
// its number of lanes) the workgroup.  Every lane gets the sum.
template <int BLOCK>
__device__ __forceinline__ float row_sum(float v, int tpr, float *red) {
    for (int o = (BLOCK ? 64 : tpr) >> 1; o >= 1; o >>= 1) v += __shfl_xor(v, o);
    if (BLOCK) {
        __syncthreads();  // the previous sum's readers
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
        for (unsigned w = 0; w < blockDim.x >> 6; ++w) v += red[w];
    }
    return v;
}

template <class T, int VE, int NV, int BLOCK>
__global__ void __launch_bounds__(BLOCK ? BLOCK : 256) norm_fwd_kernel(NormArgs a, int tpr) {
    __shared__ float red[16];
    const int D = static_cast<int>(a.D), l = BLOCK ? threadIdx.x : threadIdx.x % tpr;
    const int rows = BLOCK ? 1 : blockDim.x / tpr;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * rows + (BLOCK ? 0 : threadIdx.x / tpr);
    const bool live = row < a.rows;
    const T *x = static_cast<const T *>(a.x) + (live ? row : 0) * D;
    const float inv = 1.f / D;
    float v[NV][VE], s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        load_pack<T, VE>(x, live ? (i * tpr + l) * VE : D, D, v[i]);
#pragma unroll
        for (int e = 0; e < VE; ++e) s += v[i][e];
    }
    const float mean = row_sum<BLOCK>(s, tpr, red) * inv;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            v[i][e] -= mean;
            s += (i * tpr + l) * VE + e < D ? v[i][e] * v[i][e] : 0.f;
        }
    const float rstd = 1.f / sqrtf(row_sum<BLOCK>(s, tpr, red) * inv + a.eps);
    if (!live) return;
    const int64_t wr = a.G > 1 ? row % a.G : 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + l) * VE;
        float w[VE], b[VE];
        load_weight<VE>(a.w, a.w_bf16, wr, c, D, 1.f, w);
        load_weight<VE>(a.b, a.w_bf16, wr, c, D, 0.f, b);
#pragma unroll
        for (int e = 0; e < VE; ++e) v[i][e] = v[i][e] * rstd * w[e] + b[e];
        store_pack<T, VE>(static_cast<T *>(a.y) + row * D, c, D, v[i]);
    }
    if (l == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

// Each lane keeps the same columns of the same weight row for all its rows
// (the launch steps by a multiple of G rows), so its shares of dw and db stay
// in registers; part[2][slots][D] takes them, slot = row slot of the launch.
template <class T, int VE, int NV, int BLOCK>
__global__ void __launch_bounds__(BLOCK ? BLOCK : 256) norm_bwd_kernel(NormArgs a, int tpr, float *part) {
    __shared__ float red[16];
    const int D = static_cast<int>(a.D), l = BLOCK ? threadIdx.x : threadIdx.x % tpr;
    const int rows = BLOCK ? 1 : blockDim.x / tpr;
    const int64_t slot = static_cast<int64_t>(blockIdx.x) * rows + (BLOCK ? 0 : threadIdx.x / tpr);
    const int64_t slots = static_cast<int64_t>(gridDim.x) * rows, wr = a.G > 1 ? slot % a.G : 0;
    const float inv = 1.f / D;
    float w[NV][VE], dw[NV][VE], db[NV][VE];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        load_weight<VE>(a.w, a.w_bf16, wr, (i * tpr + l) * VE, D, 1.f, w[i]);
#pragma unroll
        for (int e = 0; e < VE; ++e) dw[i][e] = db[i][e] = 0.f;
    }
    // every wave of a workgroup runs the same number of rounds
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * rows; at < a.rows; at += slots) {
        const int64_t row = at + (BLOCK ? 0 : threadIdx.x / tpr);
        const bool live = row < a.rows;
        const int64_t r = live ? row : 0;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float x[NV][VE], dy[NV][VE], s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + l) * VE;
            load_pack<T, VE>(static_cast<const T *>(a.x) + r * D, live ? c : D, D, x[i]);
            load_pack<T, VE>(static_cast<const T *>(a.dy) + r * D, live ? c : D, D, dy[i]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                x[i][e] = (x[i][e] - mean) * rstd;  // xh; dy is zero outside the row
                dw[i][e] += dy[i][e] * x[i][e];
                db[i][e] += dy[i][e];
                dy[i][e] *= w[i][e];
                s1 += dy[i][e];
                s2 += dy[i][e] * x[i][e];
            }
        s1 = row_sum<BLOCK>(s1, tpr, red) * inv;
        s2 = row_sum<BLOCK>(s2, tpr, red) * inv;
        if (live) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
#pragma unroll
                for (int e = 0; e < VE; ++e) x[i][e] = rstd * (dy[i][e] - s1 - x[i][e] * s2);
                store_pack<T, VE>(static_cast<T *>(a.dx) + row * D, (i * tpr + l) * VE, D, x[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + l) * VE;
        if (a.dw) store_pack<float, VE>(part + slot * D, c, D, dw[i]);
        if (a.db) store_pack<float, VE>(part + (slots + slot) * D, c, D, db[i]);
    }
}

// dw[g] = sum of the slots that hold weight row g, in a fixed order.
__global__ void __launch_bounds__(1024) norm_weight_kernel(NormArgs a, const float *part, int64_t slots, int blocks) {
    __shared__ double red[16][64];
    const int col = threadIdx.x & 63, r = threadIdx.x >> 6;
    const int64_t g = blockIdx.x / blocks;
    const int64_t c = static_cast<int64_t>(blockIdx.x % blocks) * 64 + col;
    const bool second = blockIdx.y == 1 || !a.dw;  // db
    const float *p = part + (second ? slots * a.D : 0);
    double s = 0.0;
    if (c < a.D)
        for (int64_t i = g + r * a.G; i < slots; i += 16 * a.G) s += p[i * a.D + c];
    red[r][col] = s;
    __syncthreads();
    if (r == 0 && c < a.D) {
        for (int i = 1; i < 16; ++i) s += red[i][col];
        store_out(static_cast<float *>(second ? a.db : a.dw), g * a.D + c, static_cast<float>(s), a.w_bf16);
    }
}

__global__ void __launch_bounds__(256) norm_zero_kernel(float *p, int64_t n, int bf16) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256)
        store_out(p, i, 0.f, bf16);
}

struct Plan {
    int ve, nv, tpr;
    int block;  // lanes of a workgroup that holds one row; 0: rows within waves
    int threads;
    int rows;  // rows of a workgroup
};

// Lanes and registers of a row: as few lanes as hold it.  A wave keeps up to
// 4 vectors (16 elements without them) a lane, a workgroup of 256 lanes 32
// elements, one of 1024 lanes (half the registers a lane) 16.
Plan plan_of(const NormArgs &a, bool vec) {
    Plan p;
    p.ve = vec ? (a.bf16 ? 8 : 4) : 1;
    const int64_t n = (a.D + p.ve - 1) / p.ve;  // vectors of a row
    const int most = vec ? 4 : 16;
    p.block = n <= 64 * most ? 0 : a.D <= 256 * 32 ? 256 : 1024;
    if (p.block) {
        p.threads = p.tpr = p.block;
        p.rows = 1;
    } else {
        p.threads = 256;
        p.tpr = 4;
        while (p.tpr < 64 && p.tpr < n) p.tpr *= 2;
        p.rows = 256 / p.tpr;
    }
    const int64_t per = (n + p.tpr - 1) / p.tpr;
    if (vec) p.nv = per <= 1 ? 1 : per <= 2 ? 2 : per <= 4 ? 4 : 8;
    else p.nv = per <= 1 ? 1 : per <= 4 ? 4 : per <= 16 ? 16 : 32;
    return p;
}

// Workgroups of the backward: enough to fill the chip, and such that a step
// of the launch is a multiple of G rows.
int64_t bwd_grid(const NormArgs &a, const Plan &p) {
    int64_t g = a.G, r = p.rows;
    while (r) {
        const int64_t t = g % r;
        g = r;
        r = t;
    }
    const int64_t unit = a.G / g;  // G / gcd(G, rows)
    const int64_t need = (a.rows + p.rows - 1) / p.rows, want = p.threads == 1024 ? 256 : 1024;
    const int64_t n = need < want ? need : want;
    return (n + unit - 1) / unit * unit;
}

bool vector_ok(const NormArgs &a, std::initializer_list<const void *> ps) {
    bool ok = a.D % (a.bf16 ? 8 : 4) == 0;
    for (const void *p : ps) ok = ok && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
    return ok;
}

template <class T, class F>
hipError_t dispatch(const Plan &p, F go) {
    using std::integral_constant;
    auto pick = [&](auto ve, auto block) -> hipError_t {
        constexpr int VE = decltype(ve)::value, B = decltype(block)::value;
        constexpr int MOST = (B == 0 ? (VE > 1 ? 4 * VE : 16) : B == 256 ? 32 : 16) / VE;  // vectors of a lane
        hipError_t e = hipErrorInvalidValue;
        auto use = [&](auto nv) {
            if constexpr (decltype(nv)::value <= MOST) e = go(ve, nv, block);
        };
        switch (p.nv) {
            case 1: use(integral_constant<int, 1>{}); break;
            case 2: if constexpr (VE > 1) use(integral_constant<int, 2>{}); break;
            case 4: use(integral_constant<int, 4>{}); break;
            case 8: if constexpr (VE > 1) use(integral_constant<int, 8>{}); break;
            case 16: if constexpr (VE == 1) use(integral_constant<int, 16>{}); break;
            case 32: if constexpr (VE == 1) use(integral_constant<int, 32>{}); break;
        }
        return e;
    };
    auto vec = [&](auto block) { return p.ve > 1 ? pick(integral_constant<int, sizeof(T) == 2 ? 8 : 4>{}, block) : pick(integral_constant<int, 1>{}, block); };
    if (p.block == 1024) return vec(integral_constant<int, 1024>{});
    if (p.block == 256) return vec(integral_constant<int, 256>{});
    return vec(integral_constant<int, 0>{});
}

template <class T>
hipError_t fwd(const NormArgs &a, hipStream_t s) {
    const Plan p = plan_of(a, vector_ok(a, {a.x, a.y}));
    const int64_t grid = (a.rows + p.rows - 1) / p.rows;
    if (grid > 0x7fffffffLL) return hipErrorInvalidValue;
    return dispatch<T>(p, [&](auto ve, auto nv, auto block) {
        hipLaunchKernelGGL((norm_fwd_kernel<T, decltype(ve)::value, decltype(nv)::value, decltype(block)::value>),
                           dim3(static_cast<unsigned>(grid)), dim3(p.threads), 0, s, a, p.tpr);
        return hipGetLastError();
    });
}

template <class T>
hipError_t bwd(const NormArgs &a, float *part, hipStream_t s) {
    const Plan p = plan_of(a, vector_ok(a, {a.x, a.dy, a.dx}));
    const int64_t grid = bwd_grid(a, p), slots = grid * p.rows;
    hipError_t e = dispatch<T>(p, [&](auto ve, auto nv, auto block) {
        hipLaunchKernelGGL((norm_bwd_kernel<T, decltype(ve)::value, decltype(nv)::value, decltype(block)::value>),
                           dim3(static_cast<unsigned>(grid)), dim3(p.threads), 0, s, a, p.tpr, part);
        return hipGetLastError();
    });
    if (e != hipSuccess || (!a.dw && !a.db)) return e;
    const int blocks = static_cast<int>((a.D + 63) / 64);
    if (a.G * blocks > 0x7fffffffLL) return hipErrorInvalidValue;
    hipLaunchKernelGGL(norm_weight_kernel, dim3(static_cast<unsigned>(a.G * blocks), a.dw && a.db ? 2 : 1), dim3(1024), 0, s,
                       a, part, slots, blocks);
    return hipGetLastError();
}

}  // namespace

size_t norm_bwd_workspace(const NormArgs &a) {
    // the larger of the two ways a row may be held
    size_t most = 0;
    for (bool vec : {false, true}) {
        const Plan p = plan_of(a, vec);
        const size_t n = static_cast<size_t>(bwd_grid(a, p) * p.rows * a.D) * 8;
        most = n > most ? n : most;
    }
    return most;
}

hipError_t launch_norm_zero(void *p, int64_t n, int bf16, hipStream_t s) {
    const int64_t blocks = (n + 255) / 256;
    hipLaunchKernelGGL(norm_zero_kernel, dim3(static_cast<unsigned>(blocks < 1024 ? blocks : 1024)), dim3(256), 0, s,
                       static_cast<float *>(p), n, bf16);
    return hipGetLastError();
}

hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t s) { return a.bf16 ? fwd<uint16_t>(a, s) : fwd<float>(a, s); }
hipError_t launch_norm_bwd(const NormArgs &a, void *ws, hipStream_t s) {
    return a.bf16 ? bwd<uint16_t>(a, static_cast<float *>(ws), s) : bwd<float>(a, static_cast<float *>(ws), s);
}

}  // namespace gdn2
