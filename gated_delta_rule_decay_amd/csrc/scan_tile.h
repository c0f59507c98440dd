// scan_tile.h -- tiles of the gated scan and the chains that they form
// (scan_fwd.hip, scan_bwd.hip; scan.hip prepares a launch).
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
#pragma once

#include <type_traits>

#include "common.h"
#include "elements.h"
#include "scan.h"

namespace gdn2 {
namespace scan {

constexpr int CW = 64;  // channels of a workgroup: a wave's lanes in the joint
constexpr int ROWS = SCAN_MARK;
static_assert(ROWS == 128, "tiles are marks");
constexpr int STRIDE = 16;  // tiles from state to state
constexpr int GROUPS = 8;   // counters, each for every 8th chain: one for all would serialise the workgroups' starts
constexpr uint64_t NOT_YET = ~uint64_t(0);

// What the workgroups of a launch share, in the workspace.
struct Chain {
    int *seq;            // packed: [T + 2], 1 + the sequence index of token t at t + 1, 0 outside
    unsigned *counters;  // [GROUPS] at 64-byte steps, then the word that ends all waits
    uint64_t *maps;      // [chains][tiles][CW]
    uint64_t *states;    // [chains][tiles / STRIDE][CW]
    int tiles, chains, groups;
};
constexpr int COUNTER_STEP = 16, COUNTER_WORDS = COUNTER_STEP * (GROUPS + 1);

// Lays the shared part of a launch out in `ws` and fills it; `from` and `to`:
// what empty sequences pass through.
hipError_t prepare(const ScanArgs &a, void *ws, const float *from, float *to, Chain &ch, hipStream_t s);

// Workgroups: one a tile where chains are one tile long, else as many as run
// at once; those that start late find nothing left.
inline int grid_of(const Chain &ch, int at_once) {
    const int64_t per = (ch.chains + ch.groups - 1) / ch.groups * static_cast<int64_t>(ch.tiles);  // of a group, at most
    const int64_t most = ch.tiles > 1 ? at_once / ch.groups : per;
    return static_cast<int>((per < most ? per : most) * ch.groups);
}

inline bool aligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// What the gates hold and what a token adds: compiled in (bit 0: complement,
// bit 1: logits), or for ANY asked at run time, where a lane has registers for
// all four.
constexpr int ANY = -1;
// f(x's type, the gate's type, channels of a lane, form) of a request
template <class F>
hipError_t by_kind(const ScanArgs &a, bool vec, F f) {
    using B = uint16_t;
    auto forms = [&](auto t, auto g) {
        if (!vec) return f(t, g, std::integral_constant<int, 1>(), std::integral_constant<int, ANY>());
        const std::integral_constant<int, 8> eight;
        switch (2 * (a.logits != 0) + (a.comp != 0)) {
            case 0: return f(t, g, eight, std::integral_constant<int, 0>());
            case 1: return f(t, g, eight, std::integral_constant<int, 1>());
            case 2: return f(t, g, eight, std::integral_constant<int, 2>());
            default: return f(t, g, eight, std::integral_constant<int, 3>());
        }
    };
    if (a.bf16) return a.gate_bf16 ? forms(B(), B()) : forms(B(), float());
    return a.gate_bf16 ? forms(float(), B()) : forms(float(), float());
}

namespace {

// A workgroup's lanes: VE channels of K neighbouring tokens each.
template <int VE, int N>
struct Lanes {
    static constexpr int NTH = VE > 1 ? N : 1024;
    static constexpr int LPR = CW / VE;          // lanes of a row
    static constexpr int GRP = NTH / LPR;        // groups of rows
    static constexpr int K = ROWS / GRP;         // rows of a group
    static constexpr int PARTS = NTH / CW;       // waves; each composes
    static constexpr int PER = GRP / PARTS;      // groups, and looks back at
    static constexpr int LOOK = STRIDE / PARTS;  // tiles
};

// The form, compiled in or from the request.
template <int FORM>
struct Form {
    bool comp, logits;
    __device__ __forceinline__ explicit Form(const ScanArgs &a)
        : comp(FORM == ANY ? a.comp != 0 : (FORM & 1) != 0), logits(FORM == ANY ? a.logits != 0 : (FORM & 2) != 0) {}
};

// A decay a and its complement w = 1 - a in one float: the smaller one, which
// is known to its last bits, with the sign set where it is w.  The other is its
// difference from 1, rounded once; near a = 1, where memories are long, an
// error of a counts once for each token that they span.
__device__ __forceinline__ float decay_of(float v) {
    return __float_as_int(v) < 0 ? 1.f - fabsf(v) : v;
}
__device__ __forceinline__ float rest_of(float v) {
    return __float_as_int(v) < 0 ? fabsf(v) : 1.f - v;
}

// From l = log a: w is the series of -expm1(l) for l > -0.35 (the first term
// left out is below 2^-30 of it).
__device__ __forceinline__ float small_of_log(float l) {
    const float s = 1.f + l * (1.f / 2 + l * (1.f / 6 + l * (1.f / 24 + l * (1.f / 120 + l * (1.f / 720 + l * (1.f / 5040 + l * (1.f / 40320)))))));
    const float x = __builtin_amdgcn_exp2f(l * 1.4426950408889634f);
    // bits chosen by a mask: of a ?: the compiler makes a branch for each element
    const unsigned near = -static_cast<unsigned>(l > -0.35f);
    return __uint_as_float((near & (__float_as_uint(l * s) | 0x80000000u)) | (~near & __float_as_uint(x)));
}
// From a logit g, log a = -softplus(g): a = sigmoid(-g), w = sigmoid(g).
__device__ __forceinline__ float small_of_logit(float g) {
    const float e = __builtin_amdgcn_exp2f(-fabsf(g) * 1.4426950408889634f);
    return copysignf(e * __builtin_amdgcn_rcpf(1.f + e), g);
}

// The next tile of a workgroup, in the order in which its counter gives them
// out, or -1 behind the last.
__device__ __forceinline__ int next_tile(const Chain &ch, bool start) {
    const int group = blockIdx.x % ch.groups;
    const int mine = (ch.chains - group + ch.groups - 1) / ch.groups;  // chains of the group
    unsigned i;
    if (ch.tiles > 1) i = __hip_atomic_fetch_add(ch.counters + group * COUNTER_STEP, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    else i = start ? blockIdx.x / ch.groups : INT32_MAX;
    const unsigned step = i / mine;
    return step < static_cast<unsigned>(ch.tiles) ? step * ch.chains + group + ch.groups * (i - step * mine) : -1;
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

// N words, waited for together by all lanes of a wave; those not wanted read as
// (1, 0).
template <int N>
__device__ __forceinline__ void await(const Chain &ch, const uint64_t *const (&p)[N], const bool (&want)[N], float2 (&v)[N]) {
    uint64_t w[N];
    unsigned *end = ch.counters + GROUPS * COUNTER_STEP;
    for (int spin = 0;; ++spin) {
        bool there = true;
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = __hip_atomic_load(p[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
        for (int i = 0; i < N; ++i) there = there && (!want[i] || w[i] != NOT_YET);
        if (__builtin_amdgcn_ballot_w64(!there) == 0) break;
        // over a hundred times what a launch takes: the workspace is not this call's alone
        if (spin > (1 << 18)) __hip_atomic_store(end, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if ((spin & 255) == 255 &&
            __builtin_amdgcn_readfirstlane(__hip_atomic_load(end, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)))
            break;
        __builtin_amdgcn_s_sleep(1);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = want[i] ? word(w[i]) : make_float2(1.f, 0.f);
}

// The map of the tiles of `chain` between the last state and step `i` of it
// (lane: channel jc, part jp of them), and for part 0 that state itself, or
// `start` before there is one.  (The first tile's map holds the state that the
// chain starts from, and no factor: state_out may be state0, and what a later
// tile stores there comes after the first one's read.)
template <int LOOK>
__device__ __forceinline__ float2 look_back(const Chain &ch, int64_t chain, int i, int jc, int jp, float start, float &h) {
    const int n = i % STRIDE, base = i - n;
    const uint64_t *maps = ch.maps + (chain * ch.tiles + base) * CW, *states = ch.states + (chain * (ch.tiles / STRIDE) + base / STRIDE - 1) * CW;
    const uint64_t *p[LOOK + 1];
    bool want[LOOK + 1];
    float2 v[LOOK + 1];
#pragma unroll
    for (int k = 0; k < LOOK; ++k) {
        want[k] = jp * LOOK + k < n;
        p[k] = maps + ((want[k] ? jp * LOOK + k : 0) * CW + jc);
    }
    want[LOOK] = jp == 0 && base > 0;
    p[LOOK] = want[LOOK] ? states + jc : maps + jc;
    await<LOOK + 1>(ch, p, want, v);
    h = base > 0 ? v[LOOK].y : start;
    float2 m = make_float2(1.f, 0.f);
#pragma unroll
    for (int k = 0; k < LOOK; ++k) m = make_float2(v[k].x * m.x, v[k].x * m.y + v[k].y);
    return m;
}

// No lane of the kernels branches by itself while a tile is in registers: what
// a lane does not need goes to NOWHERE, and branches are those of whole waves.

// VE elements of a row as stored.
template <class E, int VE>
struct Row {
    static constexpr int BYTES = VE * sizeof(E);
    static constexpr int N = BYTES < 16 ? 1 : BYTES / 16;  // loads
    typename std::conditional<VE == 1, E, u32x4>::type p[N];
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t b, unsigned at) {
        if constexpr (VE > 1) {
#pragma unroll
            for (int i = 0; i < N; ++i) p[i] = __builtin_amdgcn_raw_buffer_load_b128(b, at + 16 * i, 0, 0);
        } else if constexpr (sizeof(E) == 2) {
            p[0] = __builtin_amdgcn_raw_buffer_load_b16(b, at, 0, 0);
        } else {
            p[0] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, at, 0, 0));
        }
    }
    __device__ __forceinline__ float operator[](int e) const {
        if constexpr (VE == 1) return to_f32<E>(p[0]);
        else if constexpr (sizeof(E) == 2) return __uint_as_float(e & 1 ? p[0][e / 2] & 0xffff0000u : p[0][e / 2] << 16);
        else return __uint_as_float(p[e / 4][e % 4]);
    }
};

template <class E, int VE>
__device__ __forceinline__ void store_row(__amdgpu_buffer_rsrc_t b, unsigned at, const float (&v)[VE]) {
    if constexpr (VE == 1) {
        if constexpr (sizeof(E) == 2) __builtin_amdgcn_raw_buffer_store_b16(from_f32<E>(v[0]), b, at, 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[0]), b, at, 0, 0);
    } else {
#pragma unroll
        for (int i = 0; i < Row<E, VE>::N; ++i) {
            u32x4 t;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (sizeof(E) == 2) t[e] = from_f32<E>(v[2 * e]) | static_cast<unsigned>(from_f32<E>(v[2 * e + 1])) << 16;
                else t[e] = __float_as_uint(v[4 * i + e]);
            }
            __builtin_amdgcn_raw_buffer_store_b128(t, b, at + 16 * i, 0, 0);
        }
    }
}

// Where a tile is.
struct Spot {
    int step;       // of its chain
    int64_t chain, sequence;
    int64_t row;    // its first token, in the tensors
    int rows, cb;   // tokens of the sequence (the axis) from it on, up to ROWS; first channel
    int64_t mark;   // its row of the marks
};
template <bool PACKED>
__device__ __forceinline__ Spot spot_of(const Chain &ch, int64_t T, int blocks, int tile, bool back) {
    Spot p;
    p.step = static_cast<int>(static_cast<unsigned>(tile) / static_cast<unsigned>(ch.chains));
    const int chain = tile - p.step * ch.chains, q = PACKED ? 0 : static_cast<int>(static_cast<unsigned>(chain) / static_cast<unsigned>(blocks));
    p.chain = chain;
    p.sequence = q;
    p.cb = (chain - q * blocks) * CW;
    const int64_t i = back ? ch.tiles - 1 - p.step : p.step;
    p.row = q * T + i * ROWS;
    p.rows = static_cast<int>(T - i * ROWS < ROWS ? T - i * ROWS : ROWS);
    p.mark = static_cast<int64_t>(q) * ch.tiles + i;
    return p;
}

// What a lane's rows are: 1 + their sequence (0: outside, or behind the end),
// and of the rows before and behind them.  Not packed: the first and the last
// row of a sequence are no edges, its states enter and leave with the chain.
template <int K, bool PACKED>
struct Rows {
    int sq[K + 2];
    bool edges;  // in any lane of the wave
    __device__ __forceinline__ void read(const int *seq, int64_t row, int r0, int rows) {
        if constexpr (PACKED) {
            const auto b = buffer<int>(seq, row, rows + 2);
#pragma unroll
            for (int k = 0; k < K + 2; ++k) sq[k] = __builtin_amdgcn_raw_buffer_load_b32(b, (r0 + k) * 4, 0, 0);
            bool edge = false;
#pragma unroll
            for (int k = 0; k < K; ++k) edge = edge || first(k) || last(k);
            edges = __builtin_amdgcn_ballot_w64(edge) != 0;
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k) sq[k + 1] = r0 + k < rows;
            edges = false;
        }
    }
    __device__ __forceinline__ bool live(int k) const { return sq[k + 1] != 0; }
    __device__ __forceinline__ bool first(int k) const { return PACKED && live(k) && sq[k] != sq[k + 1]; }
    __device__ __forceinline__ bool last(int k) const { return PACKED && live(k) && sq[k + 2] != sq[k + 1]; }
    // offset of the row's sequence in states [N, D] for a channel's byte offset, or nowhere
    __device__ __forceinline__ unsigned state(int k, bool on, unsigned D, unsigned c4) const {
        return on ? static_cast<unsigned>(sq[k + 1] - 1) * (D * 4) + c4 : NOWHERE;
    }
};

// The next tile's number, for all lanes of wave 0; other waves get nothing.
__device__ __forceinline__ int take(const Chain &ch, bool start) {
    int t = 0;
    if (threadIdx.x == 0) t = next_tile(ch, start);
    return t;
}

}  // namespace
}  // namespace scan
}  // namespace gdn2
