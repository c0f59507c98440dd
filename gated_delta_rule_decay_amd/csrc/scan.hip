// scan.hip -- a gated linear recurrence over channels, forward and backward.
//
//   h_t = a_t h_{t-1} + w_t x_t                    w = 1 or 1 - a
//   r_t = a_t (dy_t + r_{t+1})                     r from the last token back
//   dx_t = w_t (dy_t + r_{t+1}),  d log a_t = r_t (h_{t-1} - [w = 1 - a] x_t)
//
// A token is the affine map h -> a h + u of a channel's state, and maps
// compose: (a2, u2) after (a1, u1) is (a2 a1, a2 u1 + u2).  The work is cut into
// tiles of 128 tokens and 64 channels.  A lane of a workgroup holds 32 elements
// of a tile (8 channels of 4 tokens, or 1 of 32), composes its tokens, and the
// groups' maps are composed over LDS; the state that enters the tile comes from
// the tiles before it, and the lane then runs its tokens once more.  So every
// element is read once.
//
// Between tiles (a chain: the tiles of one block of channels of one sequence):
// a tile leaves its map, and every 16th tile the state behind it, as one 64-bit
// word a channel, both halves and the fact that it is there in one store.  A
// tile composes the up to 15 maps since the last such state, always the same
// ones in the same order, so that results do not depend on the timing.  A
// workgroup takes its tiles from a counter, tokens ascending, and a tile waits
// only for tiles that the counter gave out before it, so for workgroups that
// already run: the wait ends.  (It is bounded all the same, for calls that
// share a workspace at the same time, which is not allowed.)
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

constexpr int STRIDE = 16;   // tiles from state to state
constexpr int LOOK = STRIDE / (NTH / CW);  // tiles that a lane looks back at
constexpr int GROUPS = 8;    // counters, each for every 8th chain: one for all would serialise the workgroups' starts
constexpr uint64_t NOT_YET = ~uint64_t(0);

// What the workgroups of a launch share, in the workspace.
struct Chain {
    int *seq;            // sequence index of each token, packed sequences only
    unsigned *counters;  // [GROUPS] at 64-byte steps, then the word that ends all waits
    uint64_t *maps;      // [chains][tiles][CW]
    uint64_t *states;    // [chains][tiles / STRIDE][CW]
    int tiles, chains, groups;
};
constexpr int COUNTER_STEP = 16, COUNTER_WORDS = COUNTER_STEP * (GROUPS + 1);

// Before a launch: the shared words, the sequence index of each token (-1
// outside), and the states of empty sequences, which pass through.
__global__ void __launch_bounds__(256) scan_plan_kernel(Chain ch, int64_t words, const int32_t *cu, int n, int T, int D,
                                                       const float *from, float *to) {
    const int64_t step = static_cast<int64_t>(gridDim.x) * 256, first = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (ch.tiles > 1) {
        if (first < COUNTER_WORDS) ch.counters[first] = 0;
        for (int64_t i = first; i < words; i += step) ch.maps[i] = NOT_YET;
    }
    if (!cu) return;
    for (int64_t t = first; t < T; t += step) {
        int lo = 0, hi = n;  // the last sequence that starts at or before t
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= t) lo = mid + 1;
            else hi = mid;
        }
        ch.seq[t] = lo > 0 && t < cu[lo] ? lo - 1 : -1;
    }
    if (!to) return;
    for (int64_t i = first; i < static_cast<int64_t>(n) * D; i += step) {
        const int q = static_cast<int>(i / D);
        const int lo = min(max(cu[q], 0), T), hi = min(max(cu[q + 1], lo), T);
        if (hi == lo && to != from) to[i] = from ? from[i] : 0.f;
    }
}

// The next tile of a workgroup, in the order in which its counter gives them
// out, or -1 behind the last.
__device__ __forceinline__ int64_t next_tile(const Chain &ch, bool start) {
    const int group = blockIdx.x % ch.groups;
    const int mine = (ch.chains - group + ch.groups - 1) / ch.groups;  // chains of the group
    int64_t i;
    if (ch.tiles > 1) i = __hip_atomic_fetch_add(ch.counters + group * COUNTER_STEP, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    else i = start ? blockIdx.x / ch.groups : INT32_MAX;
    const int64_t tile = i / mine;
    return tile < ch.tiles ? tile * ch.chains + group + ch.groups * (i - tile * mine) : -1;
}

// A channel's word: (factor, addend) of a map, or (anything, state).
__device__ __forceinline__ void leave(uint64_t *p, float a, float u) {
    unsigned hi = __float_as_uint(u);
    if (hi == 0xffffffffu) hi = 0x7fc00000u;  // a NaN like any other: NOT_YET stays apart
    __hip_atomic_store(p, static_cast<uint64_t>(hi) << 32 | __float_as_uint(a), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 word(uint64_t w) {
    return make_float2(__uint_as_float(static_cast<unsigned>(w)), __uint_as_float(static_cast<unsigned>(w >> 32)));
}

// N words, waited for together; those not wanted read as (1, 0).
template <int N>
__device__ __forceinline__ void await(const Chain &ch, const uint64_t *const (&p)[N], const bool (&want)[N], float2 (&v)[N]) {
    uint64_t w[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        w[i] = want[i] ? __hip_atomic_load(p[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : static_cast<uint64_t>(0x3f800000u);
    unsigned *end = ch.counters + GROUPS * COUNTER_STEP;
    for (int spin = 0;; ++spin) {
        bool there = true;
#pragma unroll
        for (int i = 0; i < N; ++i) there = there && w[i] != NOT_YET;
        if (there) break;
        // over a hundred times what a launch takes: the workspace is not this call's alone
        if (spin > (1 << 18)) __hip_atomic_store(end, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if ((spin & 255) == 255 && __hip_atomic_load(end, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) break;
        __builtin_amdgcn_s_sleep(1);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (w[i] == NOT_YET) w[i] = __hip_atomic_load(p[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = word(w[i]);
}

// The map of the tiles of `chain` between the last state and step `i` of it
// (lane: channel jc, part jp of them), and for part 0 that state itself, or
// `start` before there is one.  (The first tile's map holds the state that the
// chain starts from, and no factor: state_out may be state0, and what a later
// tile stores there comes after the first one's read.)
__device__ __forceinline__ float2 look_back(const Chain &ch, int64_t chain, int i, int jc, int jp, float start, float &h) {
    const int n = i % STRIDE, base = i - n;
    const uint64_t *p[LOOK + 1];
    bool want[LOOK + 1];
    float2 v[LOOK + 1];
#pragma unroll
    for (int k = 0; k < LOOK; ++k) {
        const int at = jp * LOOK + k;
        want[k] = at < n;
        p[k] = ch.maps + ((chain * ch.tiles + base + (want[k] ? at : 0)) * CW + jc);
    }
    want[LOOK] = jp == 0 && base > 0;
    p[LOOK] = ch.states + ((chain * (ch.tiles / STRIDE) + (want[LOOK] ? base / STRIDE - 1 : 0)) * CW + jc);
    await<LOOK + 1>(ch, p, want, v);
    h = base > 0 ? v[LOOK].y : start;
    float2 m = make_float2(1.f, 0.f);
#pragma unroll
    for (int k = 0; k < LOOK; ++k) m = make_float2(v[k].x * m.x, v[k].x * m.y + v[k].y);
    return m;
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
__global__ void __launch_bounds__(NTH, VE > 1 ? 3 : 1) scan_fwd_kernel(ScanArgs a, Chain ch) {
    using Q = Tile<T, G, VE>;
    constexpr int K = Q::K, PARTS = NTH / CW;
    __shared__ float2 s_map[Q::GROUPS][CW];  // groups' maps, then .y the state that enters
    __shared__ float2 s_part[PARTS][CW], s_look[PARTS][CW];
    __shared__ float s_start[CW];
    __shared__ int64_t s_tile;
    const int blocks = static_cast<int>((a.D + CW - 1) / CW);
    const int l = threadIdx.x % Q::LPR, g = threadIdx.x / Q::LPR;
    const int jc = threadIdx.x % CW, jp = threadIdx.x / CW;  // channel and part of the joint
    const int64_t T0 = a.T;

    if (threadIdx.x == 0) s_tile = next_tile(ch, true);
    __syncthreads();
    for (int64_t tile = s_tile; tile >= 0;) {
        const int64_t step = tile / ch.chains, chain = tile - step * ch.chains;
        const int64_t sequence = PACKED ? 0 : chain / blocks;
        const int cb = static_cast<int>(chain - (PACKED ? 0 : sequence * blocks)) * CW;
        const int64_t c = cb + l * VE, t0 = step * ROWS + g * K;
        const bool col = c < a.D, jcol = cb + jc < a.D;
        const T *x = static_cast<const T *>(a.x) + sequence * T0 * a.D;
        const G *gate = static_cast<const G *>(a.gate) + sequence * T0 * a.D;
        T *y = static_cast<T *>(a.y) + sequence * T0 * a.D;
        float *marks = a.marks ? a.marks + sequence * ch.tiles * a.D : nullptr;
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
            if (PACKED && t < T0) sq[k] = ch.seq[t];
        }
        int64_t next = 0;
        if (threadIdx.x == 0) next = next_tile(ch, false);
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
            if (PACKED && sq[k] >= 0 && (t == 0 || ch.seq[t - 1] != sq[k])) {  // a sequence's first token
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
        float h0 = 0.f, h = 0.f;
        if (!PACKED && step == 0 && jp == 0 && a.s0 && jcol) h0 = a.s0[sequence * a.D + cb + jc];
        __syncthreads();
        if (threadIdx.x == 0) s_tile = next;
        {
            float2 m = make_float2(1.f, 0.f);
            for (int i = 0; i < Q::PER; ++i) {
                const float2 n = s_map[jp * Q::PER + i][jc];
                m = make_float2(n.x * m.x, n.x * m.y + n.y);
            }
            s_part[jp][jc] = m;
        }
        __syncthreads();
        tile = s_tile;
        if (ch.tiles > 1) {
            if (jp == 0 && step + 1 < ch.tiles) {
                float2 m = s_part[0][jc];
                for (int i = 1; i < PARTS; ++i) m = make_float2(s_part[i][jc].x * m.x, s_part[i][jc].x * m.y + s_part[i][jc].y);
                if (step == 0) m = make_float2(0.f, m.x * h0 + m.y);  // the later tiles do not read state0
                leave(ch.maps + (chain * ch.tiles + step) * CW + jc, m.x, m.y);
            }
            s_look[jp][jc] = look_back(ch, chain, static_cast<int>(step), jc, jp, h0, h);
            if (jp == 0) s_start[jc] = h;
            __syncthreads();
            h = s_start[jc];
            for (int i = 0; i < PARTS; ++i) h = s_look[i][jc].x * h + s_look[i][jc].y;
        } else {
            if (jp == 0) s_start[jc] = h0;
            __syncthreads();
            h = s_start[jc];
        }
        for (int i = 0; i < jp; ++i) h = s_part[i][jc].x * h + s_part[i][jc].y;
        for (int i = 0; i < Q::PER; ++i) {
            float2 &m = s_map[jp * Q::PER + i][jc];
            const float next_h = m.x * h + m.y;
            m.y = h;
            h = next_h;
        }
        if (jp == PARTS - 1 && step % STRIDE == STRIDE - 1 && step + 1 < ch.tiles)
            leave(ch.states + (chain * (ch.tiles / STRIDE) + step / STRIDE) * CW + jc, 0.f, h);
        __syncthreads();
        float hv[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) hv[e] = s_map[g][l * VE + e].y;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t t = t0 + k;
            const bool live = col && sq[k] >= 0;
            if (marks && t % ROWS == 0 && live && !(PACKED && (t == 0 || ch.seq[t - 1] != sq[k]))) {
#pragma unroll
                for (int e = 0; e < VE; ++e) marks[t / ROWS * a.D + c + e] = hv[e];
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) hv[e] = A[k][e] * hv[e] + U[k][e];
            if (live) {
                store_row<T, VE>(y + t * a.D + c, hv);
                if (a.s_out && (t == T0 - 1 || (PACKED && ch.seq[t + 1] != sq[k]))) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) a.s_out[(PACKED ? sq[k] : sequence) * a.D + c + e] = hv[e];
                }
            }
        }
    }
}

template <class T, class G, int VE, bool PACKED>
__global__ void __launch_bounds__(NTH, VE > 1 ? 2 : 1) scan_bwd_kernel(ScanArgs a, Chain ch) {
    using Q = Tile<T, G, VE>;
    constexpr int K = Q::K, PARTS = NTH / CW;
    __shared__ float2 s_map[Q::GROUPS][CW], s_rev[Q::GROUPS][CW];
    __shared__ float2 s_part[PARTS][CW], s_rpart[PARTS][CW], s_look[PARTS][CW];
    __shared__ float s_start[CW];
    __shared__ int64_t s_tile;
    const int blocks = static_cast<int>((a.D + CW - 1) / CW);
    const int l = threadIdx.x % Q::LPR, g = threadIdx.x / Q::LPR;
    const int jc = threadIdx.x % CW, jp = threadIdx.x / CW;
    const int64_t T0 = a.T;

    if (threadIdx.x == 0) s_tile = next_tile(ch, true);
    __syncthreads();
    for (int64_t tile = s_tile; tile >= 0;) {
        // steps of a chain go from its last tile to its first
        const int64_t step = tile / ch.chains, chain = tile - step * ch.chains, at = ch.tiles - 1 - step;
        const int64_t sequence = PACKED ? 0 : chain / blocks;
        const int cb = static_cast<int>(chain - (PACKED ? 0 : sequence * blocks)) * CW;
        const int64_t c = cb + l * VE, t0 = at * ROWS + g * K;
        const bool col = c < a.D, jcol = cb + jc < a.D;
        const int64_t off = sequence * T0 * a.D;
        const T *x = static_cast<const T *>(a.x) + off, *dy = static_cast<const T *>(a.dy) + off;
        const G *gate = static_cast<const G *>(a.gate) + off;
        T *dx = static_cast<T *>(a.dx) + off;
        G *dg = static_cast<G *>(a.d_gate) + off;
        // the state that enters the tile, and the gradient that enters the chain
        float h = jcol ? a.marks[(sequence * ch.tiles + at) * a.D + cb + jc] : 0.f, r0 = 0.f, r = 0.f;
        if (!PACKED && step == 0 && jp == 0 && a.d_sT && jcol) r0 = a.d_sT[sequence * a.D + cb + jc];
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
                sq[k] = ch.seq[t];
                first[k] = sq[k] >= 0 && (t == 0 || ch.seq[t - 1] != sq[k]);
                last[k] = sq[k] >= 0 && (t == T0 - 1 || ch.seq[t + 1] != sq[k]);
            }
        }
        int64_t next = 0;
        if (threadIdx.x == 0) next = next_tile(ch, false);
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
        if (threadIdx.x == 0) s_tile = next;
        {
            float2 m = make_float2(1.f, 0.f), n = make_float2(1.f, 0.f);
            for (int i = 0; i < Q::PER; ++i) {
                const float2 p = s_map[jp * Q::PER + i][jc], q = s_rev[jp * Q::PER + i][jc];
                m = make_float2(p.x * m.x, p.x * m.y + p.y);
                n = make_float2(n.x * q.x, n.x * q.y + n.y);
            }
            s_part[jp][jc] = m;
            s_rpart[jp][jc] = n;
        }
        __syncthreads();
        tile = s_tile;
        if (ch.tiles > 1) {
            if (jp == 0 && step + 1 < ch.tiles) {
                float2 n = s_rpart[0][jc];
                for (int i = 1; i < PARTS; ++i) n = make_float2(n.x * s_rpart[i][jc].x, n.x * s_rpart[i][jc].y + n.y);
                if (step == 0) n = make_float2(0.f, n.x * r0 + n.y);
                leave(ch.maps + (chain * ch.tiles + step) * CW + jc, n.x, n.y);
            }
            s_look[jp][jc] = look_back(ch, chain, static_cast<int>(step), jc, jp, r0, r);
            if (jp == 0) s_start[jc] = r;
            __syncthreads();
            r = s_start[jc];
            for (int i = 0; i < PARTS; ++i) r = s_look[i][jc].x * r + s_look[i][jc].y;
        } else {
            if (jp == 0) s_start[jc] = r0;
            __syncthreads();
            r = s_start[jc];
        }
        for (int i = 0; i < jp; ++i) h = s_part[i][jc].x * h + s_part[i][jc].y;
        for (int i = PARTS - 1; i > jp; --i) r = s_rpart[i][jc].x * r + s_rpart[i][jc].y;
        for (int i = 0; i < Q::PER; ++i) {
            float2 &m = s_map[jp * Q::PER + i][jc];
            const float next_h = m.x * h + m.y;
            m.y = h;
            h = next_h;
        }
        for (int i = Q::PER - 1; i >= 0; --i) {
            float2 &m = s_rev[jp * Q::PER + i][jc];
            const float next_r = m.x * r + m.y;
            m.y = r;
            r = next_r;
        }
        if (jp == 0 && step % STRIDE == STRIDE - 1 && step + 1 < ch.tiles)
            leave(ch.states + (chain * (ch.tiles / STRIDE) + step / STRIDE) * CW + jc, 0.f, r);
        __syncthreads();
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
                for (int e = 0; e < VE; ++e) a.d_s0[(PACKED ? sq[k] : sequence) * a.D + c + e] = rv[e];
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
int64_t tiles_of(const ScanArgs &a) { return (a.T + ROWS - 1) / ROWS; }
size_t align256(size_t n) { return (n + 255) / 256 * 256; }

size_t seq_bytes(const ScanArgs &a) { return a.cu ? align256(static_cast<size_t>(a.T) * 4) : 0; }
int64_t words_of(const ScanArgs &a) {
    const int64_t tiles = tiles_of(a);
    return tiles > 1 ? chains_of(a) * (tiles + tiles / STRIDE) * CW : 0;
}

// The shared part of a launch, laid out in `ws` and filled; `from` and `to`:
// what empty sequences pass through.
hipError_t prepare(const ScanArgs &a, void *ws, const float *from, float *to, Chain &ch, hipStream_t s) {
    char *p = static_cast<char *>(ws);
    ch.tiles = static_cast<int>(tiles_of(a));
    ch.chains = static_cast<int>(chains_of(a));
    ch.groups = ch.chains < GROUPS ? ch.chains : GROUPS;
    ch.seq = reinterpret_cast<int *>(p);
    p += seq_bytes(a);
    ch.counters = reinterpret_cast<unsigned *>(p);
    p += align256(COUNTER_WORDS * 4);
    ch.maps = reinterpret_cast<uint64_t *>(p);
    ch.states = ch.maps + static_cast<int64_t>(ch.chains) * ch.tiles * CW;
    const int64_t words = words_of(a);
    if (!a.cu && !words) return hipSuccess;
    int64_t work = a.cu ? a.T : 0;
    if (a.cu && to && a.N * a.D > work) work = a.N * a.D;
    if (words > work) work = words;
    if (work < COUNTER_WORDS) work = COUNTER_WORDS;
    work = (work + 255) / 256;
    hipLaunchKernelGGL(scan_plan_kernel, dim3(static_cast<unsigned>(work < 2048 ? work : 2048)), dim3(256), 0, s, ch, words, a.cu,
                       static_cast<int>(a.N), static_cast<int>(a.T), static_cast<int>(a.D), from, to);
    return hipGetLastError();
}

// Workgroups: one a tile where chains are one tile long, else as many as run
// at once; those that start late find nothing left.
int grid_of(const Chain &ch, int at_once) {
    const int64_t per = (ch.chains + ch.groups - 1) / ch.groups * static_cast<int64_t>(ch.tiles);  // of a group, at most
    const int64_t most = ch.tiles > 1 ? at_once / ch.groups : per;
    return static_cast<int>((per < most ? per : most) * ch.groups);
}

}  // namespace

bool scan_fits(const ScanArgs &a) {
    const int64_t tiles = tiles_of(a) > 0 ? tiles_of(a) : 1, blocks = (a.D + CW - 1) / CW;
    return blocks <= (INT64_C(1) << 24) / (a.cu || a.N == 0 ? 1 : a.N) && chains_of(a) < (INT64_C(1) << 24) &&
           chains_of(a) <= INT32_MAX / tiles;
}

size_t scan_workspace(const ScanArgs &a) {
    const int64_t words = words_of(a);
    return seq_bytes(a) + (words ? align256(COUNTER_WORDS * 4) + static_cast<size_t>(words) * 8 : 0);
}

hipError_t launch_scan_fwd(const ScanArgs &a, void *ws, hipStream_t s) {
    Chain ch = {};
    const hipError_t e = prepare(a, ws, a.s0, a.s_out, ch, s);
    if (e != hipSuccess) return e;
    const bool vec = a.D % 8 == 0 && aligned(a.x) && aligned(a.gate) && aligned(a.y);
    return by_type(a.bf16, a.gate_bf16, [&](auto t, auto g) {
        using T = decltype(t);
        using G = decltype(g);
        const dim3 grid(grid_of(ch, 768));
        auto go = [&](auto k) { hipLaunchKernelGGL(k, grid, dim3(NTH), 0, s, a, ch); };
        if (vec) a.cu ? go(scan_fwd_kernel<T, G, 8, true>) : go(scan_fwd_kernel<T, G, 8, false>);
        else a.cu ? go(scan_fwd_kernel<T, G, 1, true>) : go(scan_fwd_kernel<T, G, 1, false>);
        return hipGetLastError();
    });
}

hipError_t launch_scan_bwd(const ScanArgs &a, void *ws, hipStream_t s) {
    Chain ch = {};
    const hipError_t e = prepare(a, ws, a.d_sT, a.d_s0, ch, s);
    if (e != hipSuccess) return e;
    const bool vec = a.D % 8 == 0 && aligned(a.x) && aligned(a.gate) && aligned(a.dy) && aligned(a.dx) && aligned(a.d_gate);
    return by_type(a.bf16, a.gate_bf16, [&](auto t, auto g) {
        using T = decltype(t);
        using G = decltype(g);
        const dim3 grid(grid_of(ch, 512));
        auto go = [&](auto k) { hipLaunchKernelGGL(k, grid, dim3(NTH), 0, s, a, ch); };
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
