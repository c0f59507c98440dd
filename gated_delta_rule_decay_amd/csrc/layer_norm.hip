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
// across workgroups fp64).  Measured, bf16, whole calls in a warm loop: forward
// 524288 x 128 rows 56 us (4.8 TB/s, the rate of a large copy), backward 32768
// x 2048 with dw and db 86 us (4.7 TB/s).  The figures at the launch rules
// below are of replayed graphs on two inputs in turn.
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
struct alignas(VE * sizeof(T) < 16 ? VE * sizeof(T) : 16) Pack {
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
// the weight's elements at columns c .. (bf16 or fp32), `none` without one
template <int VE>
__device__ __forceinline__ void load_weight(const void *w, int w_bf16, int64_t row, int c, int D, float none, float (&v)[VE]) {
#pragma unroll
    for (int e = 0; e < VE; ++e) v[e] = none;
    if (!w || c >= D) return;
    if (w_bf16) load_pack<uint16_t, VE>(static_cast<const uint16_t *>(w) + row * D, c, D, v);
    else load_pack<float, VE>(static_cast<const float *>(w) + row * D, c, D, v);
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

// Raw elements of a row as this lane holds them, so that the next row's loads
// are in flight while a row is summed.
template <class T, int VE, int NV>
struct Row {
    Pack<T, VE> p[NV];
    __device__ __forceinline__ void load(const T *x, int l, int tpr, int D) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + l) * VE;
            if (c < D) p[i] = *reinterpret_cast<const Pack<T, VE> *>(x + c);
            else p[i] = Pack<T, VE>{};
        }
    }
    __device__ __forceinline__ float at(int i, int e) const { return to_f32<T>(p[i].e[e]); }
};

// Each lane keeps the same columns of the same weight row for all its rows
// (the launch steps by a multiple of G rows), so the weight is read once.
template <class T, int VE, int NV, int BLOCK>
__global__ void __launch_bounds__(BLOCK ? BLOCK : 256) norm_fwd_kernel(NormArgs a, int tpr) {
    __shared__ float red[16];
    const int D = static_cast<int>(a.D), l = BLOCK ? threadIdx.x : threadIdx.x % tpr;
    const int rows = BLOCK ? 1 : blockDim.x / tpr;
    const int64_t slot = static_cast<int64_t>(blockIdx.x) * rows + (BLOCK ? 0 : threadIdx.x / tpr);
    const int64_t step = static_cast<int64_t>(gridDim.x) * rows, wr = a.G > 1 ? slot % a.G : 0;
    const float inv = 1.f / D;
    const T *x = static_cast<const T *>(a.x);
    Row<T, VE, NV> cur, next;
    // lanes past the last row read row 0 and store nothing
    cur.load(x + (slot < a.rows ? slot : 0) * D, l, tpr, D);
    float w[NV][VE], b[NV][VE];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        load_weight<VE>(a.w, a.w_bf16, wr, (i * tpr + l) * VE, D, 1.f, w[i]);
        load_weight<VE>(a.b, a.w_bf16, wr, (i * tpr + l) * VE, D, 0.f, b[i]);
    }
    // every wave of a workgroup runs the same number of rounds
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * rows, row = slot; at < a.rows; at += step, row += step) {
        if (at + step < a.rows) next.load(x + (row + step < a.rows ? row + step : 0) * D, l, tpr, D);
        float v[NV][VE], s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                v[i][e] = cur.at(i, e);
                s += v[i][e];
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
        if (row < a.rows) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
#pragma unroll
                for (int e = 0; e < VE; ++e) v[i][e] = v[i][e] * rstd * w[i][e] + b[i][e];
                store_pack<T, VE>(static_cast<T *>(a.y) + row * D, (i * tpr + l) * VE, D, v[i]);
            }
            if (l == 0) {
                if (a.mean) a.mean[row] = mean;
                if (a.rstd) a.rstd[row] = rstd;
            }
        }
        cur = next;
    }
}

// As the forward; a lane's shares of dw and db stay in registers over all its
// rows.  With one weight row for all, a workgroup adds its lanes' shares up
// and stores one row of part[2][gridDim][D]; else every row slot stores its
// own, part[2][gridDim * rows][D].
template <class T, int VE, int NV, int BLOCK>
__global__ void __launch_bounds__(BLOCK ? BLOCK : 256) norm_bwd_kernel(NormArgs a, int tpr, float *part) {
    constexpr bool AHEAD = BLOCK != 1024;  // half the registers a lane: no room for a second row
    __shared__ float red[16];
    extern __shared__ float share[];  // [4][D] (rows within waves, one weight row)
    const int D = static_cast<int>(a.D), l = BLOCK ? threadIdx.x : threadIdx.x % tpr;
    const int rows = BLOCK ? 1 : blockDim.x / tpr;
    const int64_t slot = static_cast<int64_t>(blockIdx.x) * rows + (BLOCK ? 0 : threadIdx.x / tpr);
    const int64_t step = static_cast<int64_t>(gridDim.x) * rows, wr = a.G > 1 ? slot % a.G : 0;
    const float inv = 1.f / D;
    const T *x = static_cast<const T *>(a.x), *dy = static_cast<const T *>(a.dy);
    Row<T, VE, NV> cx, cy, nx, ny;
    float mean, rstd, next_mean = 0.f, next_rstd = 0.f;
    {
        const int64_t r = slot < a.rows ? slot : 0;
        cx.load(x + r * D, l, tpr, D);
        cy.load(dy + r * D, l, tpr, D);
        mean = a.mean[r];
        rstd = a.rstd[r];
    }
    float w[NV][VE], dw[NV][VE], db[NV][VE];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        load_weight<VE>(a.w, a.w_bf16, wr, (i * tpr + l) * VE, D, 1.f, w[i]);
#pragma unroll
        for (int e = 0; e < VE; ++e) dw[i][e] = db[i][e] = 0.f;
    }
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * rows, row = slot; at < a.rows; at += step, row += step) {
        if (AHEAD && at + step < a.rows) {
            const int64_t r = row + step < a.rows ? row + step : 0;
            nx.load(x + r * D, l, tpr, D);
            ny.load(dy + r * D, l, tpr, D);
            next_mean = a.mean[r];
            next_rstd = a.rstd[r];
        }
        const bool live = row < a.rows;
        float h[NV][VE], g[NV][VE], s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float d = live ? cy.at(i, e) : 0.f;  // zero outside the row too
                h[i][e] = live ? (cx.at(i, e) - mean) * rstd : 0.f;
                dw[i][e] += d * h[i][e];
                db[i][e] += d;
                g[i][e] = d * w[i][e];
                s1 += g[i][e];
                s2 += g[i][e] * h[i][e];
            }
        s1 = row_sum<BLOCK>(s1, tpr, red) * inv;
        s2 = row_sum<BLOCK>(s2, tpr, red) * inv;
        if (live) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
#pragma unroll
                for (int e = 0; e < VE; ++e) h[i][e] = rstd * (g[i][e] - s1 - h[i][e] * s2);
                store_pack<T, VE>(static_cast<T *>(a.dx) + row * D, (i * tpr + l) * VE, D, h[i]);
            }
        }
        if (AHEAD) {
            cx = nx;
            cy = ny;
            mean = next_mean;
            rstd = next_rstd;
        } else if (row + step < a.rows) {
            cx.load(x + (row + step) * D, l, tpr, D);
            cy.load(dy + (row + step) * D, l, tpr, D);
            mean = a.mean[row + step];
            rstd = a.rstd[row + step];
        }
    }
    if (!BLOCK && a.G == 1) {
        const int wave = threadIdx.x >> 6;
        for (int which = 0; which < 2; ++which) {
            if (!(which ? a.db : a.dw)) continue;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float v[VE];
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    v[e] = which ? db[i][e] : dw[i][e];
                    for (int o = tpr; o < 64; o <<= 1) v[e] += __shfl_xor(v[e], o);
                    const int c = (i * tpr + l) * VE + e;
                    if ((threadIdx.x & 63) < static_cast<unsigned>(tpr) && c < D) share[wave * D + c] = v[e];
                }
            }
            __syncthreads();
            float *p = part + (which * static_cast<int64_t>(gridDim.x) + blockIdx.x) * D;
            for (int c = threadIdx.x; c < D; c += 256) p[c] = (share[c] + share[D + c]) + (share[2 * D + c] + share[3 * D + c]);
            __syncthreads();
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + l) * VE;
        if (a.dw) store_pack<float, VE>(part + slot * D, c, D, dw[i]);
        if (a.db) store_pack<float, VE>(part + (step + slot) * D, c, D, db[i]);
    }
}

// dw[g] = sum of the slots that hold weight row g, in a fixed order.  A
// workgroup takes 16 columns, 64 lanes each a share of the slots.
__global__ void __launch_bounds__(1024) norm_weight_kernel(NormArgs a, const float *part, int64_t slots, int blocks) {
    __shared__ double red[16][16];
    const int col = threadIdx.x & 15, r = threadIdx.x >> 4, wave = threadIdx.x >> 6;
    const int64_t g = blockIdx.x / blocks;
    const int64_t c = static_cast<int64_t>(blockIdx.x % blocks) * 16 + col;
    const bool second = blockIdx.y == 1 || !a.dw;  // db
    const float *p = part + (second ? slots * a.D : 0) + c;
    double s = 0.0;
    if (c < a.D) {
        int64_t i = g + r * a.G;
        for (; i + 192 * a.G < slots; i += 256 * a.G) {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = p[(i + 64 * k * a.G) * a.D];
            s += static_cast<double>(v[0]) + v[1] + v[2] + v[3];
        }
        for (; i < slots; i += 64 * a.G) s += p[i * a.D];
    }
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if ((threadIdx.x & 63) < 16) red[wave][col] = s;
    __syncthreads();
    if (threadIdx.x < 16 && c < a.D) {
        s = 0.0;
        for (int i = 0; i < 16; ++i) s += red[i][col];
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

// Vectors that a lane of a row within a wave holds at most.  Forward: with 2,
// wider rows go to a workgroup each (32768 x 2048 bf16: 53 us, with 4 in a
// wave 56; 64 rows: 4.2 and 5.4).  Backward: 4 (89 us, with 2 93).
constexpr int FWD_WAVE = 2, BWD_WAVE = 4;

// Lanes and registers of a row: as few lanes as hold it, since the sums over
// a workgroup cost two barriers each and those of 1024 lanes most (16384 x
// 4096 bf16 forward: 54 us with 256 lanes, 97 with 1024).  256 lanes hold up
// to 32 elements each, backward 16 where they are vectors (8192 x 8192 bf16:
// 138 us with 256 lanes of 32 elements, 118 with 1024 of 8; 16384 x 4096: 90
// with 256 of 16, 158 with 1024), 1024 lanes (half the registers) 16.
Plan plan_of(const NormArgs &a, bool vec, bool backward) {
    Plan p;
    p.ve = vec ? (a.bf16 ? 8 : 4) : 1;
    const int64_t n = (a.D + p.ve - 1) / p.ve;  // vectors of a row
    const int most = !vec ? 16 : backward ? BWD_WAVE : FWD_WAVE;
    p.block = n <= 64 * most ? 0 : a.D <= 256 * (vec && backward ? 16 : 32) ? 256 : 1024;
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

// Workgroups of a launch: up to `want`, and such that a step of the launch is
// a multiple of G rows.
int64_t grid_of(const NormArgs &a, const Plan &p, int64_t want) {
    int64_t g = a.G, r = p.rows;
    while (r) {
        const int64_t t = g % r;
        g = r;
        r = t;
    }
    const int64_t unit = a.G / g;  // G / gcd(G, rows)
    const int64_t need = (a.rows + p.rows - 1) / p.rows;
    const int64_t n = need < want ? need : want;
    return (n + unit - 1) / unit * unit;
}
int64_t fwd_grid(const NormArgs &a, const Plan &p) { return grid_of(a, p, p.threads == 1024 ? 256 : 2048); }
// Backward: as many workgroups as run at once, for 256 CUs.  A second round
// of a few more leaves most CUs idle, and every workgroup adds partial sums.
// What runs at once follows from the registers that the elements of a lane
// take: up to 8 elements four a CU (524288 x 128 bf16: 85 us, three 91), 16
// three (65536 x 1024: 84, four 102; 16384 x 4096: 90, four 115), without
// vectors two (65536 x 509 fp32: 103, three 128), 32 two in waves (32768 x
// 2048: 89, three 103, four 96), one over a workgroup (4096 x 8191: 99, two
// 115), and one of 1024 lanes (8192 x 8192: 118, two 121).
int64_t bwd_grid(const NormArgs &a, const Plan &p) {
    const int held = p.ve * p.nv;
    const int per_cu = p.block == 1024 ? 1 : held <= 8 ? 4 : held <= 16 ? (p.ve > 1 ? 3 : 2) : p.block ? 1 : 2;
    return grid_of(a, p, 256 * per_cu);
}

// rows of the partial sums
int64_t slots_of(const NormArgs &a, const Plan &p) {
    return bwd_grid(a, p) * (a.G == 1 ? 1 : p.rows);
}

bool vector_ok(const NormArgs &a, std::initializer_list<const void *> ps) {
    bool ok = a.D % (a.bf16 ? 8 : 4) == 0;
    for (const void *p : ps) ok = ok && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
    return ok;
}

template <class T, int WAVE, class F>
hipError_t dispatch(const Plan &p, F go) {
    using std::integral_constant;
    auto pick = [&](auto ve, auto block) -> hipError_t {
        constexpr int VE = decltype(ve)::value, B = decltype(block)::value;
        constexpr int MOST = (B == 0 ? (VE > 1 ? WAVE * VE : 16) : B == 256 ? (VE > 1 && WAVE == BWD_WAVE ? 16 : 32) : 16) / VE;  // vectors of a lane
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
    const Plan p = plan_of(a, vector_ok(a, {a.x, a.y, a.w, a.b}), false);
    const int64_t grid = fwd_grid(a, p);
    if (grid > 0x7fffffffLL) return hipErrorInvalidValue;
    return dispatch<T, FWD_WAVE>(p, [&](auto ve, auto nv, auto block) {
        hipLaunchKernelGGL((norm_fwd_kernel<T, decltype(ve)::value, decltype(nv)::value, decltype(block)::value>),
                           dim3(static_cast<unsigned>(grid)), dim3(p.threads), 0, s, a, p.tpr);
        return hipGetLastError();
    });
}

template <class T>
hipError_t bwd(const NormArgs &a, float *part, hipStream_t s) {
    const Plan p = plan_of(a, vector_ok(a, {a.x, a.dy, a.dx, a.w}), true);
    const int64_t grid = bwd_grid(a, p), slots = slots_of(a, p);
    const size_t lds = !p.block && a.G == 1 ? 4 * a.D * sizeof(float) : 0;
    hipError_t e = dispatch<T, BWD_WAVE>(p, [&](auto ve, auto nv, auto block) {
        hipLaunchKernelGGL((norm_bwd_kernel<T, decltype(ve)::value, decltype(nv)::value, decltype(block)::value>),
                           dim3(static_cast<unsigned>(grid)), dim3(p.threads), lds, s, a, p.tpr, part);
        return hipGetLastError();
    });
    if (e != hipSuccess || (!a.dw && !a.db)) return e;
    const int blocks = static_cast<int>((a.D + 15) / 16);
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
        const Plan p = plan_of(a, vec, true);
        const size_t n = static_cast<size_t>(slots_of(a, p) * a.D) * 8;
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
