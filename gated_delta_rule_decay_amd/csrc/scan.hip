// scan.hip -- a gated linear recurrence over channels, forward and backward.
//
//   h_t = a_t h_{t-1} + w_t x_t                    w = 1 or 1 - a
//   r_t = a_t (dy_t + r_{t+1})                     r from the last token back
//   dx_t = w_t (dy_t + r_{t+1}),  d log a_t = r_t (h_{t-1} - [w = 1 - a] x_t)
//
// A token is the affine map h -> a h + u of a channel's state, and maps
// compose: (a2, u2) after (a1, u1) is (a2 a1, a2 u1 + u2).  A workgroup takes
// 64 channels and walks over tiles of 128 tokens.  A lane holds 32 elements of
// a tile (8 channels of 4 tokens, or 1 of 32), composes its tokens, and the
// groups' maps are composed over LDS in a fixed order, which gives every group
// the state that enters it; the lane then runs its tokens once more.  So a tile
// is read once, and its result does not depend on the launch.
//
// Packed sequences are one axis with resets: at a sequence's first token the
// state comes from state0, (0, a s0 + u), and backward the gradient that enters
// a sequence's last token from behind is d_state_out's.  What a token is comes
// from a table of sequence indices, one a token, built on the device.
#include <type_traits>

#include "common.h"
#include "elements.h"
#include "scan.h"

namespace gdn2 {
namespace {

constexpr int NTH = 256;  // 4 waves
constexpr int CW = 64;    // channels of a workgroup
constexpr int ROWS = SCAN_MARK;
static_assert(ROWS == 128, "tiles are marks");

template <class T>
__device__ __forceinline__ T from_f32(float x) {
    if constexpr (sizeof(T) == 2) return f32_to_bf16(x);
    else return x;
}

// a = exp(l) and w = 1 - a.  Near 0, where memories are long and an error of a
// counts once for each token that they span, w is the series of -expm1(l) (the
// first term left out is below 2^-30 of it) and a = 1 - w, rounded once.
__device__ __forceinline__ void decay_of(float l, float &a, float &w) {
    const float s = 1.f + l * (1.f / 2 + l * (1.f / 6 + l * (1.f / 24 + l * (1.f / 120 + l * (1.f / 720 + l * (1.f / 5040 + l * (1.f / 40320)))))));
    const float p = -l * s, x = __builtin_amdgcn_exp2f(l * 1.4426950408889634f);
    const bool near = l > -0.35f;
    w = near ? p : 1.f - x;
    a = near ? 1.f - p : x;
}

// log a = -softplus(g): a = sigmoid(-g), w = sigmoid(g), the smaller one from
// the exponential, the other as its difference from 1, rounded once.
__device__ __forceinline__ void decay_of_logit(float g, float &a, float &w) {
    const float e = __builtin_amdgcn_exp2f(-fabsf(g) * 1.4426950408889634f);
    const float small = e * __builtin_amdgcn_rcpf(1.f + e), big = 1.f - small;
    a = g >= 0.f ? small : big;
    w = g >= 0.f ? big : small;
}

// In place: gates F (as stored) to decays a; W = 1 - a.
template <int K, int VE>
__device__ __forceinline__ void both_gates(int logits, float (&F)[K][VE], float (&W)[K][VE]) {
    auto all = [&](auto f) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                float d;
                f(F[k][e], d, W[k][e]);
                F[k][e] = d;
            }
    };
    if (logits) all([](float x, float &d, float &w) { decay_of_logit(x, d, w); });
    else all([](float x, float &d, float &w) { decay_of(x, d, w); });
}

// Sequence index of each token, -1 outside; and the states of empty sequences,
// which pass through.
__global__ void __launch_bounds__(256) scan_plan_kernel(const int32_t *cu, int n, int T, int D, int *seq, const float *from,
                                                       float *to) {
    const int64_t step = static_cast<int64_t>(gridDim.x) * 256, first = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    for (int64_t t = first; t < T; t += step) {
        int lo = 0, hi = n;  // the last sequence that starts at or before t
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= t) lo = mid + 1;
            else hi = mid;
        }
        seq[t] = lo > 0 && t < cu[lo] ? lo - 1 : -1;
    }
    if (!to) return;
    for (int64_t i = first; i < static_cast<int64_t>(n) * D; i += step) {
        const int q = static_cast<int>(i / D);
        const int lo = min(max(cu[q], 0), T), hi = min(max(cu[q + 1], lo), T);
        if (hi == lo && to != from) to[i] = from ? from[i] : 0.f;
    }
}

// A lane's share of a tile: 32 elements.
template <class T, class G, int VE>
struct Tile {
    static constexpr int LPR = CW / VE;          // lanes of a row
    static constexpr int GROUPS = NTH / LPR;     // groups of rows
    static constexpr int K = ROWS / GROUPS;      // rows of a group
    static constexpr int PER = GROUPS / (NTH / CW);  // groups that a lane of the joint composes
};

template <class E, int VE>
__device__ __forceinline__ void load_row(const E *p, bool on, float (&v)[VE]) {
    if constexpr (VE == 1) {
        v[0] = on ? to_f32<E>(*p) : 0.f;
    } else {
        constexpr int N = 16 / sizeof(E);  // elements of 16 bytes
#pragma unroll
        for (int i = 0; i < VE; i += N) {
            Pack<E, N> t = {};
            if (on) t = *reinterpret_cast<const Pack<E, N> *>(p + i);
#pragma unroll
            for (int e = 0; e < N; ++e) v[i + e] = to_f32<E>(t.e[e]);
        }
    }
}

template <class E, int VE>
__device__ __forceinline__ void store_row(E *p, const float (&v)[VE]) {
    if constexpr (VE == 1) {
        *p = from_f32<E>(v[0]);
    } else {
        constexpr int N = 16 / sizeof(E);
#pragma unroll
        for (int i = 0; i < VE; i += N) {
            Pack<E, N> t;
#pragma unroll
            for (int e = 0; e < N; ++e) t.e[e] = from_f32<E>(v[i + e]);
            *reinterpret_cast<Pack<E, N> *>(p + i) = t;
        }
    }
}

template <class T, class G, int VE, bool PACKED>
__global__ void __launch_bounds__(NTH) scan_fwd_kernel(ScanArgs a, const int *seq) {
    using Q = Tile<T, G, VE>;
    constexpr int K = Q::K;
    __shared__ float2 s_map[Q::GROUPS][CW];  // groups' maps, then .y the state that enters
    __shared__ float2 s_part[NTH / CW][CW];
    __shared__ float s_carry[CW];
    const int blocks = static_cast<int>((a.D + CW - 1) / CW);
    const int64_t chain = blockIdx.x / blocks;
    const int cb = (blockIdx.x % blocks) * CW, l = threadIdx.x % Q::LPR, g = threadIdx.x / Q::LPR;
    const int64_t c = cb + l * VE;
    const bool col = c < a.D;
    const int jc = threadIdx.x % CW, jp = threadIdx.x / CW;  // channel and part of the joint
    const int64_t T0 = a.T;
    const T *x = static_cast<const T *>(a.x) + chain * T0 * a.D;
    const G *gate = static_cast<const G *>(a.gate) + chain * T0 * a.D;
    T *y = static_cast<T *>(a.y) + chain * T0 * a.D;
    float *marks = a.marks ? a.marks + chain * ((T0 + ROWS - 1) / ROWS) * a.D : nullptr;
    if (threadIdx.x < CW) s_carry[jc] = !PACKED && a.s0 && cb + jc < a.D ? a.s0[chain * a.D + cb + jc] : 0.f;

    for (int64_t base = 0; base < T0; base += ROWS) {
        const int64_t t0 = base + g * K;
        float A[K][VE], U[K][VE], ca[VE], cu[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            ca[e] = 1.f;
            cu[e] = 0.f;
        }
        int sq[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t t = t0 + k;
            const bool on = col && t < T0;
            load_row<T, VE>(x + t * a.D + c, on, U[k]);
            load_row<G, VE>(gate + t * a.D + c, on, A[k]);
            sq[k] = t < T0 ? 0 : -1;
            if (PACKED && t < T0) sq[k] = seq[t];
        }
        {
            float W[K][VE];
            both_gates<K, VE>(a.logits, A, W);
            if (a.comp)
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int e = 0; e < VE; ++e) U[k][e] *= W[k][e];
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t t = t0 + k;
            if (PACKED && sq[k] >= 0 && (t == 0 || seq[t - 1] != sq[k])) {  // a sequence's first token
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float h0 = a.s0 && col ? a.s0[sq[k] * a.D + c + e] : 0.f;
                    // here, not below: another wave may end this sequence, and state_out may be state0
                    if (marks && t % ROWS == 0 && col) marks[t / ROWS * a.D + c + e] = h0;
                    U[k][e] += A[k][e] * h0;
                    A[k][e] = 0.f;
                }
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                if (sq[k] < 0) {
                    A[k][e] = 1.f;
                    U[k][e] = 0.f;
                }
                cu[e] = A[k][e] * cu[e] + U[k][e];
                ca[e] *= A[k][e];
            }
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) s_map[g][l * VE + e] = make_float2(ca[e], cu[e]);
        __syncthreads();
        {
            float pa = 1.f, pu = 0.f;
            for (int i = 0; i < Q::PER; ++i) {
                const float2 m = s_map[jp * Q::PER + i][jc];
                pu = m.x * pu + m.y;
                pa *= m.x;
            }
            s_part[jp][jc] = make_float2(pa, pu);
        }
        __syncthreads();
        float h = s_carry[jc];
        for (int i = 0; i < jp; ++i) h = s_part[i][jc].x * h + s_part[i][jc].y;
        for (int i = 0; i < Q::PER; ++i) {
            float2 &m = s_map[jp * Q::PER + i][jc];
            const float next = m.x * h + m.y;
            m.y = h;
            h = next;
        }
        __syncthreads();
        if (jp == NTH / CW - 1) s_carry[jc] = h;  // read after the next tile's barriers
        float hv[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) hv[e] = s_map[g][l * VE + e].y;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t t = t0 + k;
            const bool live = col && sq[k] >= 0;
            if (marks && t % ROWS == 0 && live && !(PACKED && (t == 0 || seq[t - 1] != sq[k]))) {
#pragma unroll
                for (int e = 0; e < VE; ++e) marks[t / ROWS * a.D + c + e] = hv[e];
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) hv[e] = A[k][e] * hv[e] + U[k][e];
            if (live) {
                store_row<T, VE>(y + t * a.D + c, hv);
                if (a.s_out && (PACKED ? t == T0 - 1 || seq[t + 1] != sq[k] : t == T0 - 1)) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) a.s_out[(PACKED ? sq[k] : chain) * a.D + c + e] = hv[e];
                }
            }
        }
    }
}

template <class T, class G, int VE, bool PACKED>
__global__ void __launch_bounds__(NTH) scan_bwd_kernel(ScanArgs a, const int *seq) {
    using Q = Tile<T, G, VE>;
    constexpr int K = Q::K;
    __shared__ float2 s_map[Q::GROUPS][CW], s_rev[Q::GROUPS][CW];
    __shared__ float2 s_part[NTH / CW][CW], s_rpart[NTH / CW][CW];
    __shared__ float s_carry[CW];
    const int blocks = static_cast<int>((a.D + CW - 1) / CW);
    const int64_t chain = blockIdx.x / blocks;
    const int cb = (blockIdx.x % blocks) * CW, l = threadIdx.x % Q::LPR, g = threadIdx.x / Q::LPR;
    const int64_t c = cb + l * VE;
    const bool col = c < a.D;
    const int jc = threadIdx.x % CW, jp = threadIdx.x / CW;
    const bool jcol = cb + jc < a.D;
    const int64_t T0 = a.T, tiles = (T0 + ROWS - 1) / ROWS;
    const int64_t at = chain * T0 * a.D;
    const T *x = static_cast<const T *>(a.x) + at, *dy = static_cast<const T *>(a.dy) + at;
    const G *gate = static_cast<const G *>(a.gate) + at;
    T *dx = static_cast<T *>(a.dx) + at;
    G *dg = static_cast<G *>(a.d_gate) + at;
    const float *marks = a.marks + chain * tiles * a.D;
    if (threadIdx.x < CW) s_carry[jc] = !PACKED && a.d_sT && jcol ? a.d_sT[chain * a.D + cb + jc] : 0.f;

    for (int64_t base = (tiles - 1) * ROWS; base >= 0; base -= ROWS) {
        const int64_t t0 = base + g * K;
        // maps of the group: forward (fa, fu), backward (ra, ru)
        float X[K][VE], F[K][VE], W[K][VE], Y[K][VE], fa[VE], fu[VE], ra[VE], ru[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            fa[e] = ra[e] = 1.f;
            fu[e] = ru[e] = 0.f;
        }
        int sq[K];
        bool first[K], last[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t t = t0 + k;
            const bool on = col && t < T0;
            load_row<T, VE>(x + t * a.D + c, on, X[k]);
            load_row<G, VE>(gate + t * a.D + c, on, F[k]);
            load_row<T, VE>(dy + t * a.D + c, on, Y[k]);
            sq[k] = t < T0 ? 0 : -1;
            first[k] = last[k] = false;
            if (PACKED && t < T0) {
                sq[k] = seq[t];
                first[k] = sq[k] >= 0 && (t == 0 || seq[t - 1] != sq[k]);
                last[k] = sq[k] >= 0 && (t == T0 - 1 || seq[t + 1] != sq[k]);
            }
        }
        both_gates<K, VE>(a.logits, F, W);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (PACKED && last[k] && a.d_sT && col)
#pragma unroll
                for (int e = 0; e < VE; ++e) Y[k][e] += a.d_sT[sq[k] * a.D + c + e];
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                float f = F[k][e], u = a.comp ? W[k][e] * X[k][e] : X[k][e], af = f;
                if (PACKED && first[k]) {
                    if (a.s0 && col) u += f * a.s0[sq[k] * a.D + c + e];
                    af = 0.f;
                }
                if (sq[k] < 0) {
                    u = 0.f;
                    af = f = 1.f;
                    Y[k][e] = 0.f;
                }
                fu[e] = af * fu[e] + u;
                fa[e] *= af;
                // the group's map from right to left: this token's map comes before
                ru[e] += ra[e] * f * Y[k][e];
                ra[e] *= PACKED && last[k] ? 0.f : f;
            }
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            s_map[g][l * VE + e] = make_float2(fa[e], fu[e]);
            s_rev[g][l * VE + e] = make_float2(ra[e], ru[e]);
        }
        __syncthreads();
        {
            float pa = 1.f, pu = 0.f, qa = 1.f, qu = 0.f;
            for (int i = 0; i < Q::PER; ++i) {
                const float2 m = s_map[jp * Q::PER + i][jc], n = s_rev[jp * Q::PER + i][jc];
                pu = m.x * pu + m.y;
                pa *= m.x;
                qu += qa * n.y;
                qa *= n.x;
            }
            s_part[jp][jc] = make_float2(pa, pu);
            s_rpart[jp][jc] = make_float2(qa, qu);
        }
        __syncthreads();
        float h = jcol ? marks[base / ROWS * a.D + cb + jc] : 0.f, r = s_carry[jc];
        for (int i = 0; i < jp; ++i) h = s_part[i][jc].x * h + s_part[i][jc].y;
        for (int i = NTH / CW - 1; i > jp; --i) r = s_rpart[i][jc].x * r + s_rpart[i][jc].y;
        for (int i = 0; i < Q::PER; ++i) {
            float2 &m = s_map[jp * Q::PER + i][jc];
            const float next = m.x * h + m.y;
            m.y = h;
            h = next;
        }
        for (int i = Q::PER - 1; i >= 0; --i) {
            float2 &m = s_rev[jp * Q::PER + i][jc];
            const float next = m.x * r + m.y;
            m.y = r;
            r = next;
        }
        __syncthreads();
        if (jp == 0) s_carry[jc] = r;  // read after the next tile's barriers
        float H[K][VE], hv[VE], rv[VE];  // H: the states that enter the tokens
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            hv[e] = s_map[g][l * VE + e].y;
            rv[e] = s_rev[g][l * VE + e].y;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                if (PACKED && first[k]) hv[e] = a.s0 && col ? a.s0[sq[k] * a.D + c + e] : 0.f;
                H[k][e] = hv[e];
                if (sq[k] >= 0) hv[e] = F[k][e] * hv[e] + (a.comp ? W[k][e] * X[k][e] : X[k][e]);
            }
        }
#pragma unroll
        for (int k = K - 1; k >= 0; --k) {
            const int64_t t = t0 + k;
            if (sq[k] < 0 || !col) continue;
            float gx[VE], gl[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float s = Y[k][e] + (PACKED && last[k] ? 0.f : rv[e]);
                rv[e] = F[k][e] * s;
                gx[e] = a.comp ? W[k][e] * s : s;
                gl[e] = rv[e] * (H[k][e] - (a.comp ? X[k][e] : 0.f));
                if (a.logits) gl[e] *= -W[k][e];
            }
            store_row<T, VE>(dx + t * a.D + c, gx);
            store_row<G, VE>(dg + t * a.D + c, gl);
            if (a.d_s0 && (PACKED ? first[k] : t == 0)) {
#pragma unroll
                for (int e = 0; e < VE; ++e) a.d_s0[(PACKED ? sq[k] : chain) * a.D + c + e] = rv[e];
            }
        }
    }
}

template <class T, class G, int VE>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanStepArgs a) {
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * VE;
    if (i >= a.n) return;
    float x[VE], g[VE], h[VE];
    load_row<T, VE>(static_cast<const T *>(a.x) + i, true, x);
    load_row<G, VE>(static_cast<const G *>(a.gate) + i, true, g);
    load_row<float, VE>(a.state + i, true, h);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
        float f, w;
        if (a.logits) decay_of_logit(g[e], f, w);
        else decay_of(g[e], f, w);
        h[e] = f * h[e] + (a.comp ? w * x[e] : x[e]);
    }
    store_row<float, VE>(a.state + i, h);
    store_row<T, VE>(static_cast<T *>(a.y) + i, h);
}

bool aligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <class F>
hipError_t by_type(int bf16, int gate_bf16, F f) {
    using B = uint16_t;
    if (bf16) return gate_bf16 ? f(B(), B()) : f(B(), float());
    return gate_bf16 ? f(float(), B()) : f(float(), float());
}

int64_t chains_of(const ScanArgs &a) { return (a.cu ? 1 : a.N) * ((a.D + CW - 1) / CW); }

// the table of sequence indices, at the start of the workspace
hipError_t plan(const ScanArgs &a, const float *from, float *to, int *seq, hipStream_t s) {
    int64_t work = a.T > a.N * a.D && to ? a.T : to ? a.N * a.D : a.T;
    work = (work + 255) / 256;
    hipLaunchKernelGGL(scan_plan_kernel, dim3(static_cast<unsigned>(work < 2048 ? work : 2048)), dim3(256), 0, s, a.cu,
                       static_cast<int>(a.N), static_cast<int>(a.T), static_cast<int>(a.D), seq, from, to);
    return hipGetLastError();
}

}  // namespace

bool scan_fits(const ScanArgs &a) {
    const int64_t tiles = (a.T + ROWS - 1) / ROWS, most = INT32_MAX / (tiles > 0 ? tiles : 1);
    const int64_t blocks = (a.D + CW - 1) / CW;
    return blocks <= most / (a.cu || a.N == 0 ? 1 : a.N) && chains_of(a) < (INT64_C(1) << 24);
}

size_t scan_workspace(const ScanArgs &a, bool) { return a.cu ? (static_cast<size_t>(a.T) * 4 + 255) / 256 * 256 : 0; }

hipError_t launch_scan_fwd(const ScanArgs &a, void *ws, hipStream_t s) {
    int *seq = static_cast<int *>(ws);
    if (a.cu) {
        const hipError_t e = plan(a, a.s0, a.s_out, seq, s);
        if (e != hipSuccess) return e;
    }
    const bool vec = a.D % 8 == 0 && aligned(a.x) && aligned(a.gate) && aligned(a.y);
    return by_type(a.bf16, a.gate_bf16, [&](auto t, auto g) {
        using T = decltype(t);
        using G = decltype(g);
        const dim3 grid(static_cast<unsigned>(chains_of(a)));
        auto go = [&](auto k) { hipLaunchKernelGGL(k, grid, dim3(NTH), 0, s, a, seq); };
        if (vec) a.cu ? go(scan_fwd_kernel<T, G, 8, true>) : go(scan_fwd_kernel<T, G, 8, false>);
        else a.cu ? go(scan_fwd_kernel<T, G, 1, true>) : go(scan_fwd_kernel<T, G, 1, false>);
        return hipGetLastError();
    });
}

hipError_t launch_scan_bwd(const ScanArgs &a, void *ws, hipStream_t s) {
    int *seq = static_cast<int *>(ws);
    if (a.cu) {
        const hipError_t e = plan(a, a.d_sT, a.d_s0, seq, s);
        if (e != hipSuccess) return e;
    }
    const bool vec = a.D % 8 == 0 && aligned(a.x) && aligned(a.gate) && aligned(a.dy) && aligned(a.dx) && aligned(a.d_gate);
    return by_type(a.bf16, a.gate_bf16, [&](auto t, auto g) {
        using T = decltype(t);
        using G = decltype(g);
        const dim3 grid(static_cast<unsigned>(chains_of(a)));
        auto go = [&](auto k) { hipLaunchKernelGGL(k, grid, dim3(NTH), 0, s, a, seq); };
        if (vec) a.cu ? go(scan_bwd_kernel<T, G, 8, true>) : go(scan_bwd_kernel<T, G, 8, false>);
        else a.cu ? go(scan_bwd_kernel<T, G, 1, true>) : go(scan_bwd_kernel<T, G, 1, false>);
        return hipGetLastError();
    });
}

hipError_t launch_scan_step(const ScanStepArgs &a, hipStream_t s) {
    const bool vec = a.n % 8 == 0 && aligned(a.x) && aligned(a.gate) && aligned(a.y) && aligned(a.state);
    return by_type(a.bf16, a.gate_bf16, [&](auto t, auto g) {
        using T = decltype(t);
        using G = decltype(g);
        const int64_t lanes = vec ? a.n / 8 : a.n, grid = (lanes + 255) / 256;
        if (grid > INT32_MAX) return hipErrorInvalidValue;
        if (vec) hipLaunchKernelGGL((scan_step_kernel<T, G, 8>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, a);
        else hipLaunchKernelGGL((scan_step_kernel<T, G, 1>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, a);
        return hipGetLastError();
    });
}

}  // namespace gdn2
