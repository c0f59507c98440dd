// rotary.hip -- rotary positions of queries and keys, alone or behind the norm
// of each head, and the gradients of both.
//
//   turn:  u' = m (c u - s v),  v' = m (s u + c v),   c, s = cos, sin (p f_j)
//   norm:  h = x r,  y = turn(w h),  r = 1 / sqrt(mean x^2 + eps) or 1 / |x|
//   back:  g = turn^T(dy),  dw = sum g h,  e = sum_channels w g h,
//          dx = r (w g - h e n),  n = 1/d (mean) or 1 (length)
//
// Bound by HBM: a row (one head of one token) is read once and held in
// registers by L lanes of a wave, a lane two vectors of VE elements: in the
// half layout channels j and rot/2 + j, so that both members of its pairs are
// in one lane, else neighbouring ones.  A workgroup takes some tokens of q or
// of k; its lanes form each (token, pair) angle once, in LDS, for all heads.
// With 2 x 16 heads of 128 bf16 channels (a large copy: 5.0 to 5.5 TB/s): 65536 tokens
// turned in 186 us, 5.8 TB/s; 32768 normed and turned in 106 us, 5.0 TB/s,
// backward in 160 us, 5.0 TB/s.  256 tokens take 4 us on the GPU, 9 from call to
// call, which the host needs for one.
//
// Angles: p f / 2 pi from products of 106 bits, so that the farthest positions have
// their part of a turn to 2^-50 as the first ones do, the nearest quarter turn
// taken off exactly, then the Taylor series of sine and cosine on [-pi/4, pi/4] in
// fp32, whose first terms left out are below 2^-28.  Everything else is fp32, rounded once at the end; a row whose sum of
// squares leaves [2^-80, 2^100] is summed and scaled in fp64 instead, so that no
// row of finite values overflows or vanishes.
#include <type_traits>

#include "common.h"
#include "elements.h"
#include "rotary.h"

namespace gdn2 {
namespace {

constexpr int NTH = 256;
// Rows of a lane group in one go.  (65536 tokens of 2 x 16 heads of 128 channels,
// rotated: 188 us with 2, 192 with 4, 201 with 8; 32768 of them normed: 109, 115,
// 163; backward 163 with 1 or 2, 314 with 4, which spill.)
constexpr int ROUNDS = 2;
constexpr int IN_FP32 = 32;     // rows of a lane that a weight's gradient sums in fp32
constexpr int MAX_TOKENS = 16;  // tokens of a workgroup
constexpr int MAX_PAIRS = 128;

// Turns of p f / 2 pi, less whole ones: the product and what its rounding left
// out, times 1 / 2 pi to 106 bits.  (Of the product alone a position of 2^40 keeps 12
// bits of a radian.)
__device__ __forceinline__ double turns_of(double p, double f) {
#pragma clang fp contract(off)
    constexpr double INV = 0x1.45f306dc9c883p-3, REST = -0x1.6b01ec5417056p-57;  // 1 / 2 pi
    const double a = p * f, b = __builtin_fma(p, f, -a), q = a * INV;
    const double left = __builtin_fma(a, INV, -q) + (a * REST + b * INV);
    const double t = (q - rint(q)) + left;
    return t - rint(t);
}

// cos and sin of 2 pi t, |t| <= 1/2
__device__ __forceinline__ void cos_sin_turns(double t, float &c, float &s) {
    const double n = rint(4.0 * t);
    const float x = 6.283185307179586f * static_cast<float>(t - 0.25 * n), y = x * x;
    const float sn = x + x * y * (-1.f / 6 + y * (1.f / 120 + y * (-1.f / 5040 + y * (1.f / 362880))));
    const float cs = 1.f + y * (-0.5f + y * (1.f / 24 + y * (-1.f / 720 + y * (1.f / 40320 + y * (-1.f / 3628800)))));
    const int q = static_cast<int>(n) & 3;  // quarter turns
    const float a = q & 1 ? sn : cs, b = q & 1 ? cs : sn;
    c = q == 1 || q == 2 ? -a : a;
    s = q >= 2 ? -b : b;
}

// The two vectors of a lane and what they are.
struct Place {
    int c0, c1;  // channels
    int j;       // first angle, where they turn
    bool turn, live;
};

template <int VE, bool INTER>
__device__ __forceinline__ Place place_of(int v, int d, int rot) {
    const int half = rot / 2, turning = (half + VE - 1) / VE;
    Place p;
    p.turn = v < turning;
    p.j = v * VE;
    if (p.turn) {
        p.c0 = INTER ? 2 * v * VE : v * VE;
        p.c1 = INTER ? p.c0 + VE : half + p.c0;
    } else {
        p.c0 = rot + 2 * VE * (v - turning);
        p.c1 = p.c0 + VE;
    }
    p.live = p.turn || p.c0 < d;
    return p;
}

// Whether element e of the first / second vector is the lane's (VEC: whole vectors are).
template <bool INTER>
__device__ __forceinline__ bool own0(const Place &p, int e, int d, int rot) {
    return p.turn ? (INTER ? p.c0 + e < rot : p.c0 + e < rot / 2) : p.c0 + e < d;
}
template <bool INTER>
__device__ __forceinline__ bool own1(const Place &p, int e, int d, int rot) {
    return p.turn ? (INTER ? p.c1 + e < rot : p.c1 + e < rot) : p.c1 + e < d;
}

// A row's two vectors of a lane.  VEC: `b` and `at` give its first element, and
// what is not the lane's reads as zero; else `row` does.
template <class T, int VE, bool VEC, bool INTER>
struct Two {
    Pack<T, VE> a, b;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t buf, unsigned at, const T *row, const Place &p, int d, int rot, bool on) {
        if constexpr (VEC) {
            a = __builtin_bit_cast(Pack<T, VE>, __builtin_amdgcn_raw_buffer_load_b128(buf, on ? at + p.c0 * static_cast<unsigned>(sizeof(T)) : NOWHERE, 0, 0));
            b = __builtin_bit_cast(Pack<T, VE>, __builtin_amdgcn_raw_buffer_load_b128(buf, on && p.c1 < d ? at + p.c1 * static_cast<unsigned>(sizeof(T)) : NOWHERE, 0, 0));
        } else {
            a = b = Pack<T, VE>{};
            if (!on) return;
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                if (own0<INTER>(p, e, d, rot)) a.e[e] = row[p.c0 + e];
                if (own1<INTER>(p, e, d, rot)) b.e[e] = row[p.c1 + e];
            }
        }
    }
};

template <class T, int VE, bool VEC, bool INTER>
__device__ __forceinline__ void store_two(__amdgpu_buffer_rsrc_t buf, unsigned at, T *row, const Place &p, int d, int rot, bool on,
                                          const float (&a)[VE], const float (&b)[VE]) {
    if constexpr (VEC) {
        Pack<T, VE> u, v;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            u.e[e] = from_f32<T>(a[e]);
            v.e[e] = from_f32<T>(b[e]);
        }
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, u), buf, on ? at + p.c0 * static_cast<unsigned>(sizeof(T)) : NOWHERE, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), buf, on && p.c1 < d ? at + p.c1 * static_cast<unsigned>(sizeof(T)) : NOWHERE, 0, 0);
    } else {
        if (!on) return;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            if (own0<INTER>(p, e, d, rot)) row[p.c0 + e] = from_f32<T>(a[e]);
            if (own1<INTER>(p, e, d, rot)) row[p.c1 + e] = from_f32<T>(b[e]);
        }
    }
}

// The rotation of a lane's pairs.
template <int VE, bool INTER>
__device__ __forceinline__ void turn(float (&a)[VE], float (&b)[VE], const float *c, const float *s) {
    if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < VE / 2; ++i) {
            const float u = a[2 * i], v = a[2 * i + 1], x = b[2 * i], y = b[2 * i + 1];
            const float c0 = c[i], s0 = s[i], c1 = c[VE / 2 + i], s1 = s[VE / 2 + i];
            a[2 * i] = c0 * u - s0 * v;
            a[2 * i + 1] = s0 * u + c0 * v;
            b[2 * i] = c1 * x - s1 * y;
            b[2 * i + 1] = s1 * x + c1 * y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            const float u = a[e], v = b[e];
            a[e] = c[e] * u - s[e] * v;
            b[e] = s[e] * u + c[e] * v;
        }
    }
}

struct Shape {
    int lanes;      // of a row, a power of two up to 64
    int tokens[2];  // of a workgroup, for q and k
    int64_t tiles[2];
    int grid[2];    // workgroups of q and k
    unsigned by_heads[2], by_pairs;  // see quotient()
};

// n / d for n < 2^16 from m = ceil(2^32 / d), d < 2^16: m d - 2^32 < d, so the
// error n (m d - 2^32) / (2^32 d) stays below 1 / d.  d = 1: m = 0.
__device__ __forceinline__ int quotient(unsigned n, unsigned m) { return m ? __umulhi(n, m) : n; }

template <class T, int VE, bool VEC, bool INTER, int MODE>
__global__ void __launch_bounds__(NTH, MODE == ROTARY_NORM_BWD && VE > 4 ? 3 : 4) rotary_kernel(RotaryArgs a, Shape sh, float *part) {
    __shared__ float s_cos[MAX_TOKENS][MAX_PAIRS + 8], s_sin[MAX_TOKENS][MAX_PAIRS + 8];
    __shared__ double s_dw[NTH / 64][MODE == ROTARY_NORM_BWD ? 256 : 1];  // each wave's sums of dw
    const int which = blockIdx.x >= static_cast<unsigned>(sh.grid[0]);
    const int block = which ? blockIdx.x - sh.grid[0] : blockIdx.x;
    const RotaryPart pt = a.part[which];
    const int L = sh.lanes, l = threadIdx.x & (L - 1), slot = threadIdx.x / L, slots = NTH / L;
    const int d = a.d, rot = a.rot, half = rot / 2, H = pt.H, TT = sh.tokens[which];
    const Place p = place_of<VE, INTER>(l, d, rot);
    const int pairs = (half + VE - 1) / VE * VE;  // angles that some lane reads
    const float per = a.l2 ? 1.f : 1.f / d;
    const double offset = static_cast<double>(a.offset);  // exact, and so are its sums with positions

    float w0[VE], w1[VE], dw0[VE], dw1[VE];
    if constexpr (MODE != ROTARY_TURN) {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            w0[e] = w1[e] = 1.f;
            dw0[e] = dw1[e] = 0.f;
            if (pt.w && p.live) {
                if (own0<INTER>(p, e, d, rot)) w0[e] = load_qkv(pt.w, p.c0 + e, a.w_bf16);
                if (own1<INTER>(p, e, d, rot)) w1[e] = load_qkv(pt.w, p.c1 + e, a.w_bf16);
            }
        }
    }

    // The lane groups' sums of dw, joined in order and added to the wave's in 64 bits:
    // fp32 sums of a thousand equal terms were off by 1e-5 of themselves.  Each
    // channel is one lane's.
    // Joins the lane groups' sums of dw in order and adds them to the wave's, in 64
    // bits: a thousand equal terms that a lane summed in fp32 were off by 1e-5 of
    // their sum.  (32768 tokens of 2 x 16 heads of 128 take 160 us either way, from odd
    // addresses 481 for 459.)  A channel is one lane's, so that none waits for another.
    const bool sums = MODE == ROTARY_NORM_BWD && pt.dw;
    int held = 0;       // rows in dw0 and dw1
    bool fresh = true;  // nothing in s_dw yet
    auto put_away = [&] {
        int lane = threadIdx.x;
        asm volatile("" : "+v"(lane));  // places worked out here, not held over the rows
        double *at = s_dw[lane >> 6];
        const bool mine = (lane & 63) < L && p.live;
        for (int o = L; o < 64; o <<= 1)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                dw0[e] += __shfl_xor(dw0[e], o);
                dw1[e] += __shfl_xor(dw1[e], o);
            }
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            if (mine && own0<INTER>(p, e, d, rot)) at[p.c0 + e] = (fresh ? 0.0 : at[p.c0 + e]) + dw0[e];
            if (mine && own1<INTER>(p, e, d, rot)) at[p.c1 + e] = (fresh ? 0.0 : at[p.c1 + e]) + dw1[e];
            dw0[e] = dw1[e] = 0.f;
        }
        held = 0;
        fresh = false;
    };

    for (int64_t tile = block; tile < sh.tiles[which]; tile += sh.grid[which]) {
        const int t0 = static_cast<int>(tile * TT), nt = a.tokens - t0 < TT ? a.tokens - t0 : TT;
        const int rows = nt * H;
        const int64_t out = static_cast<int64_t>(t0) * H * d;  // contiguous rows
        constexpr int ALL = 0x7fffffff / sizeof(T);
        const auto bx = buffer<T>(pt.x, t0 * pt.stride, ALL), bdy = buffer<T>(pt.dy, out, ALL), by = buffer<T>(pt.y, out, ALL);
        for (int base = 0; base < rows; base += slots * ROUNDS) {
            Two<T, VE, VEC, INTER> x[ROUNDS], dy[MODE == ROTARY_NORM_BWD ? ROUNDS : 1];
            int tok[ROUNDS];
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i) {
                const int r = base + slot + i * slots;
                const bool on = r < rows && p.live;
                tok[i] = r < rows ? quotient(r, sh.by_heads[which]) : 0;
                const int at = (r - tok[i] * H) * d;
                x[i].load(bx, (tok[i] * static_cast<unsigned>(pt.stride) + at) * sizeof(T),
                          static_cast<const T *>(pt.x) + (t0 + tok[i]) * pt.stride + at, p, d, rot, on);
                if constexpr (MODE == ROTARY_NORM_BWD)
                    dy[i].load(bdy, r * d * static_cast<unsigned>(sizeof(T)), static_cast<const T *>(pt.dy) + out + r * d, p, d, rot, on);
            }
            if (base == 0) {
                __syncthreads();  // the last tile's readers
                const int first = t0 % a.period;
                for (int i = threadIdx.x; i < nt * pairs; i += NTH) {
                    const int t = quotient(i, sh.by_pairs), j = i - t * pairs;
                    int at = first + t;
                    if (at >= a.period) at = a.period < MAX_TOKENS ? at % a.period : at - a.period;
                    float c = 0.f, s = 0.f;  // behind the last pair
                    if (j < half) cos_sin_turns(turns_of(offset + (a.pos ? a.pos[at] : at), a.freq[j]), c, s);
                    s_cos[t][j] = a.cos_mag * c;
                    s_sin[t][j] = a.sin_mag * s;
                }
                __syncthreads();
            }
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i) {
                const int r = base + slot + i * slots;
                const bool on = r < rows && p.live;
                float u[VE], v[VE];
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    u[e] = to_f32<T>(x[i].a.e[e]);
                    v[e] = to_f32<T>(x[i].b.e[e]);
                }
                float rs = 0.f;
                double wide = 0.0;
                bool far = false;
                if constexpr (MODE != ROTARY_TURN) {
                    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
                    for (int e = 0; e < VE; e += 2) {
                        s0 += u[e] * u[e];
                        s1 += u[e + 1] * u[e + 1];
                        s2 += v[e] * v[e];
                        s3 += v[e + 1] * v[e + 1];
                    }
                    float ss = (s0 + s1) + (s2 + s3);
                    for (int o = L >> 1; o >= 1; o >>= 1) ss += __shfl_xor(ss, o);
                    // outside, squares of fp32 overflow, or vanish beside what they add up to
                    far = r < rows && !(ss > 0x1p-80f && ss < 0x1p100f);
                    const float m = a.l2 ? ss : ss * per + a.eps;
                    rs = __builtin_amdgcn_rsqf(m);
                    // 0: no row, whose mean is eps alone (a row that is not far has more than 2^-90)
                    rs = m > 0x1p-100f ? rs * (1.5f - 0.5f * m * rs * rs) : 0.f;
                    if (__builtin_amdgcn_ballot_w64(far) != 0) {
                        double sum = 0.0;
#pragma unroll
                        for (int e = 0; e < VE; ++e) {
                            sum += static_cast<double>(u[e]) * u[e] + static_cast<double>(v[e]) * v[e];
                            asm volatile("" : "+v"(sum));  // not all elements in 64 bits at once
                        }
                        for (int o = L >> 1; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
                        sum = a.l2 ? sum : sum / d + a.eps;
                        wide = sum == 0.0 ? 0.0 : 1.0 / sqrt(sum);  // NaN stays
#pragma unroll
                        for (int e = 0; e < VE; ++e) {
                            u[e] = far ? static_cast<float>(u[e] * wide) : u[e] * rs;
                            v[e] = far ? static_cast<float>(v[e] * wide) : v[e] * rs;
                            settle(u[e]);
                            settle(v[e]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < VE; ++e) {
                            u[e] *= rs;
                            v[e] *= rs;
                        }
                    }
                }
                const float *c = &s_cos[tok[i]][p.turn ? p.j : 0], *s = &s_sin[tok[i]][p.turn ? p.j : 0];
                if constexpr (MODE == ROTARY_NORM_BWD) {
                    float g[VE], f[VE], dot = 0.f;
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        g[e] = to_f32<T>(dy[i].a.e[e]);
                        f[e] = to_f32<T>(dy[i].b.e[e]);
                    }
                    if (p.turn) turn<VE, INTER>(g, f, c, s);
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        dw0[e] += g[e] * u[e];
                        dw1[e] += f[e] * v[e];
                        g[e] *= w0[e];
                        f[e] *= w1[e];
                        dot += g[e] * u[e] + f[e] * v[e];
                    }
                    for (int o = L >> 1; o >= 1; o >>= 1) dot += __shfl_xor(dot, o);
                    dot *= per;
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        u[e] = g[e] - u[e] * dot;
                        v[e] = f[e] - v[e] * dot;
                    }
                    if (__builtin_amdgcn_ballot_w64(far) != 0) {
#pragma unroll
                        for (int e = 0; e < VE; ++e) {
                            u[e] = far ? static_cast<float>(u[e] * wide) : u[e] * rs;
                            v[e] = far ? static_cast<float>(v[e] * wide) : v[e] * rs;
                            settle(u[e]);
                            settle(v[e]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < VE; ++e) {
                            u[e] *= rs;
                            v[e] *= rs;
                        }
                    }
                } else {
                    if constexpr (MODE == ROTARY_NORM)
#pragma unroll
                        for (int e = 0; e < VE; ++e) {
                            u[e] *= w0[e];
                            v[e] *= w1[e];
                        }
                    if (p.turn) turn<VE, INTER>(u, v, c, s);
                }
                store_two<T, VE, VEC, INTER>(by, r * d * static_cast<unsigned>(sizeof(T)), static_cast<T *>(pt.y) + out + r * d, p, d, rot, on, u, v);
            }
            if (sums && (held += ROUNDS) >= IN_FP32) put_away();
        }
    }

    if constexpr (MODE == ROTARY_NORM_BWD) {
        if (!sums) return;
        put_away();
        __syncthreads();
        for (int c = threadIdx.x; c < d; c += NTH)  // one row a workgroup
            part[static_cast<int64_t>(blockIdx.x) * d + c] = static_cast<float>((s_dw[0][c] + s_dw[1][c]) + (s_dw[2][c] + s_dw[3][c]));
    }
}

// dw of q (blockIdx.y 0) or k: the sum of its workgroups' rows in a fixed
// order.  A workgroup takes 16 channels, 64 lanes each a share of the rows.
__global__ void __launch_bounds__(1024) rotary_weight_kernel(RotaryArgs a, Shape sh, const float *part) {
    __shared__ double red[16][16];
    const int which = blockIdx.y;
    if (!a.part[which].dw) return;
    const int col = threadIdx.x & 15, r = threadIdx.x >> 4, wave = threadIdx.x >> 6, c = blockIdx.x * 16 + col;
    double s = 0.0;
    if (c < a.d) {
        const float *p = part + static_cast<int64_t>(which ? sh.grid[0] : 0) * a.d + c;
        int i = r;
        for (; i + 448 < sh.grid[which]; i += 512) {  // eight loads in flight
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = p[static_cast<int64_t>(i + 64 * k) * a.d];
#pragma unroll
            for (int k = 0; k < 8; ++k) s += v[k];
        }
        for (; i < sh.grid[which]; i += 64) s += p[static_cast<int64_t>(i) * a.d];
    }
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if ((threadIdx.x & 63) < 16) red[wave][col] = s;
    __syncthreads();
    if (threadIdx.x < 16 && c < a.d) {
        s = 0.0;
        for (int i = 0; i < 16; ++i) s += red[i][col];
        store_out(static_cast<float *>(a.part[which].dw), c, static_cast<float>(s), a.w_bf16);
    }
}

// Workgroups of a part, backward: each leaves a row of sums.  (32768 tokens of 16
// heads: 163 us, with 2048 as well, with 512 176.)
constexpr int BWD_GRID = 1024;

Shape shape_of(const RotaryArgs &a, int ve) {
    Shape sh = {};
    const int n = (a.rot / 2 + ve - 1) / ve + (a.d - a.rot + 2 * ve - 1) / (2 * ve);  // lanes with a place
    sh.lanes = 1;
    while (sh.lanes < n) sh.lanes *= 2;
    const int slots = NTH / sh.lanes, pairs = (a.rot / 2 + ve - 1) / ve * ve;
    auto inverse = [](int64_t n) { return n > 1 ? static_cast<unsigned>(((INT64_C(1) << 32) + n - 1) / n) : 0u; };
    sh.by_pairs = inverse(pairs);
    for (int i = 0; i < 2; ++i) {
        const int H = a.part[i].H;
        if (!H) continue;
        sh.by_heads[i] = inverse(H);
        int t = slots * ROUNDS / H;
        t = t < 1 ? 1 : t > MAX_TOKENS ? MAX_TOKENS : t;
        sh.tokens[i] = t;
        sh.tiles[i] = (static_cast<int64_t>(a.tokens) + t - 1) / t;
        const int64_t most = a.mode == ROTARY_NORM_BWD ? BWD_GRID : INT64_C(1) << 22;
        sh.grid[i] = static_cast<int>(sh.tiles[i] < most ? sh.tiles[i] : most);
    }
    return sh;
}

// Whether rows are whole aligned vectors: channels, pair blocks and strides in
// units of VE, every pointer on 16 bytes.  Rows that are not go element by
// element (8 x 4096 tokens of 2 x 16 heads of 128 bf16 channels from an odd
// address: rotation 231 us, with the norm 260, backward 482; aligned 93, 106 and
// 160).
bool vector_ok(const RotaryArgs &a) {
    const int ve = a.bf16 ? 8 : 4;
    if (a.d % ve || a.rot % (2 * ve)) return false;
    for (const RotaryPart &p : a.part) {
        if (!p.H) continue;
        if (p.stride % ve || p.stride >= (1 << 24)) return false;  // 31-bit offsets within a workgroup's tokens
        for (const void *x : {p.x, p.dy, const_cast<const void *>(p.y)})
            if (reinterpret_cast<uintptr_t>(x) & 15) return false;
    }
    return true;
}

template <class T, int VE, bool VEC, bool INTER, int MODE>
hipError_t go(const RotaryArgs &a, float *part, hipStream_t s) {
    const Shape sh = shape_of(a, VE);
    hipLaunchKernelGGL((rotary_kernel<T, VE, VEC, INTER, MODE>), dim3(sh.grid[0] + sh.grid[1]), dim3(NTH), 0, s, a, sh, part);
    hipError_t e = hipGetLastError();
    if (MODE != ROTARY_NORM_BWD || e != hipSuccess || (!a.part[0].dw && !a.part[1].dw)) return e;
    hipLaunchKernelGGL(rotary_weight_kernel, dim3((a.d + 15) / 16, 2), dim3(1024), 0, s, a, sh, part);
    return hipGetLastError();
}

template <class T, int VE, bool VEC>
hipError_t pick(const RotaryArgs &a, float *part, hipStream_t s) {
    if (a.inter) switch (a.mode) {
        case ROTARY_TURN: return go<T, VE, VEC, true, ROTARY_TURN>(a, part, s);
        case ROTARY_NORM: return go<T, VE, VEC, true, ROTARY_NORM>(a, part, s);
        default: return go<T, VE, VEC, true, ROTARY_NORM_BWD>(a, part, s);
    }
    switch (a.mode) {
        case ROTARY_TURN: return go<T, VE, VEC, false, ROTARY_TURN>(a, part, s);
        case ROTARY_NORM: return go<T, VE, VEC, false, ROTARY_NORM>(a, part, s);
        default: return go<T, VE, VEC, false, ROTARY_NORM_BWD>(a, part, s);
    }
}

}  // namespace

size_t rotary_bwd_workspace(const RotaryArgs &a) {
    // the larger grid of the two ways a row may be held
    size_t most = 0;
    RotaryArgs b = a;
    b.mode = ROTARY_NORM_BWD;
    for (int ve : {4, 8}) {
        const Shape sh = shape_of(b, ve);
        const size_t n = static_cast<size_t>(sh.grid[0] + sh.grid[1]) * a.d * sizeof(float);
        most = n > most ? n : most;
    }
    return most;
}

hipError_t launch_rotary(const RotaryArgs &a, void *ws, hipStream_t s) {
    float *part = static_cast<float *>(ws);
    const bool vec = vector_ok(a);
    if (a.bf16) return vec ? pick<uint16_t, 8, true>(a, part, s) : pick<uint16_t, 4, false>(a, part, s);
    return vec ? pick<float, 4, true>(a, part, s) : pick<float, 4, false>(a, part, s);
}

}  // namespace gdn2
