// scan_tile.h -- tiles of the gated scan and the chains that they form
// (scan_fwd.hip, scan_bwd.hip; scan.hip prepares a launch).
//
//   h_t = a_t h_{t-1} + w_t x_t                    w = 1 or 1 - a
//   r_t = a_t (dy_t + r_{t+1})                     r from the last token back
//   dx_t = w_t (dy_t + r_{t+1}),  d log a_t = r_t (h_{t-1} - [w = 1 - a] x_t)
//
// A token is the affine map h -> a h + u of a channel's state, and maps
// compose: (a2, u2) after (a1, u1) is (a2 a1, a2 u1 + u2).  The work is cut into
// tiles of 128 tokens and 64 channels.  A lane of a workgroup holds 8 channels
// of 4 tokens, or 1 channel of 8 or 16 (of 32, in 256 lanes, would not fit its
// registers in the backward), composes its tokens, and the groups' maps
// are composed over LDS; the state that enters the tile comes from the tiles
// before it, and the lane then runs its tokens once more.  So every element is
// read once.  Rows that are not whole aligned vectors of 8 go element by element
// (8 x 4096 tokens of 2048 bf16 channels from an odd address: forward 125 us,
// backward 232; aligned 98 and 148).
//
// Bound by HBM where there are many chains; where there are few, by how long a
// word takes from one workgroup to another, twice a tile: its run's maps, and the
// run before.  (That forward moves 405 MB in 98 us, 4.1 TB/s, the backward 673 MB
// in 148 us, 4.5 TB/s, a large copy 5.0 to 5.5 TB/s; one sequence of 65536 tokens
// takes 284 us, 3.8 TB/s, of which its waits are about a fifth.)
//
// Between tiles (a chain: the tiles of one block of channels of one sequence):
// a tile leaves its map as one 64-bit word a channel, both halves and the fact
// that it is there in one store; every 16th tile leaves the map of its run of 16
// as well, and every 256th the state behind it.  A tile composes the state, the
// up to 15 runs and the up to 15 maps since then, always the same ones in the
// same order, so that results do not depend on the timing; neither a map nor a
// run waits for a state, so a chain moves on at the tiles' own pace.  A workgroup
// takes its tiles from a counter, along the chain, works on them in that order,
// and a tile waits only for tiles that the counter gave out before it: the first
// tile that is not done is at work, and the wait ends.  (It is bounded all the
// same, for calls that share a workspace at the same time, which is not allowed.
// A word that has not come by then counts as it stands, and that is NaN in both
// halves, so what depends on it is NaN.)
//
// Packed sequences are one axis with resets: at a sequence's first token the
// state comes from state0, (-0, a s0 + u), and backward the gradient that enters
// a sequence's last token from behind is d_state_out's.  A factor of -0, which no
// other map has, takes nothing of what is before it, be it infinite, NaN or the mark
// of a row of no sequence.  What a token is comes from a table of sequence
// indices, one a token, built on the device.
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
// Tiles of a run, and from state to state.  (65536 tokens of 2048 channels with a
// state behind every 16 tiles and no runs: 337 us, with runs 296; a state that
// waits for the one before it is late for all tiles behind it.)
constexpr int RUN = 16;
constexpr int SPAN = RUN * 16;
constexpr int GROUPS = 32;      // counters, each for neighbouring chains: one for all would serialise the workgroups' starts
constexpr uint64_t NOT_YET = ~uint64_t(0);

// What the workgroups of a launch share, in the workspace.
struct Chain {
    int *seq;            // packed: [T + 2], 1 + the sequence index of token t at t + 1, 0 outside
    unsigned *counters;  // [GROUPS] at 64-byte steps, then the word that ends all waits
    uint64_t *maps;      // [chains][tiles][CW]
    uint64_t *runs;      // [chains][tiles / RUN][CW]
    uint64_t *states;    // [chains][tiles / SPAN][CW]
    int tiles, chains, groups, share;  // share: chains of a group, at most
};
constexpr int COUNTER_STEP = 16, COUNTER_WORDS = COUNTER_STEP * (GROUPS + 1);

// Lays the shared part of a launch out in `ws` and fills it; `from` and `to`:
// what empty sequences pass through.
hipError_t prepare(const ScanArgs &a, void *ws, const float *from, float *to, Chain &ch, hipStream_t s);

// Workgroups: one a tile where chains are one tile long, else as many as run
// at once; those that start late find nothing left.
inline int grid_of(const Chain &ch, int at_once) {
    const int64_t per = static_cast<int64_t>(ch.share) * ch.tiles;  // of a group, at most
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
    static constexpr int NTH = N;
    static constexpr int LPR = CW / VE;          // lanes of a row
    static constexpr int GRP = NTH / LPR;        // groups of rows
    static constexpr int K = ROWS / GRP;         // rows of a group
    static constexpr int PARTS = NTH / CW;       // waves; each composes
    static constexpr int PER = GRP / PARTS;      // groups, and looks back at
    static constexpr int LOOK = RUN / PARTS;     // tiles and at runs
    // Where channel l * VE + e of a block stands in the joint, and the channel
    // that stands at q: neighbouring lanes of a group write to neighbouring
    // places, and a row of places (ROW) is so long that groups fall on other banks.
    static constexpr int ROW = CW + (VE > 1 ? 8 : 0);
    static __device__ __forceinline__ int place(int l, int e) { return e * LPR + l; }
    static __device__ __forceinline__ int channel(int q) { return q % LPR * VE + q / LPR; }
};

// A lane's place, worked out again where it is used: what follows from it is
// otherwise held in registers, or in scratch, over all tiles.
__device__ __forceinline__ int anew(int place) {
    asm volatile("" : "+v"(place));
    return place;
}

// The form, compiled in or from the request.
template <int FORM>
struct Form {
    bool comp, logits;
    __device__ __forceinline__ explicit Form(const ScanArgs &a)
        : comp(FORM == ANY ? a.comp != 0 : (FORM & 1) != 0), logits(FORM == ANY ? a.logits != 0 : (FORM & 2) != 0) {}
};

// A decay a and its complement w = 1 - a in one float: the smaller one, with
// the sign set where it is w.  The other is its difference from 1, rounded once.
// (The smaller one is as near as its exponential: from a logarithm within some
// roundings, from a logit g within 2 |g| of them, those of g log2(e).)  Near a = 1
// the rounded a is off by much of w, always to the same side where gates do not
// change: it only multiplies states for the tokens of one lane, and what passes
// between lanes is joined by complements (Joint).
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

// The counter of a workgroup.  Every 256th runs on the same CU: it gets another
// chain, because tiles of one chain on one CU take their turns at its issue slots
// while the others of the chain wait for them (65536 tokens of 2048 channels:
// 280 us, without the shift 296).  The first 256 reach all counters.
__device__ __forceinline__ unsigned group_of(const Chain &ch) {
    return (blockIdx.x + (ch.tiles > 1 ? blockIdx.x / 256 * 11 : 0)) % ch.groups;
}
// A workgroup's next number from its counter (without counters: its own, once),
// in the first lane of a wave that asks as a whole: the others add to nowhere.
// (A branch of one lane would let the compiler move what is live around it while
// the other lanes are off.)
__device__ __forceinline__ unsigned take(const Chain &ch, bool start) {
    if (ch.tiles == 1) return start ? blockIdx.x / ch.groups : INT32_MAX;
    const auto b = buffer<unsigned>(ch.counters, group_of(ch) * COUNTER_STEP, 1);
    return __builtin_amdgcn_raw_ptr_buffer_atomic_add_i32(1, b, threadIdx.x % 64 ? NOWHERE : 0, 0, 0);
}
// The tile that a number stands for, -1 behind the last.
__device__ __forceinline__ int tile_of(const Chain &ch, unsigned i) {
    // a group's chains neighbour each other: they share lines of their rows
    // (65536 rows of 4 KB copied in tiles: 5.45 TB/s, with every 8th block of
    // channels 4.95)
    const unsigned first = group_of(ch) * ch.share, left = ch.chains - first;
    const unsigned mine = left < static_cast<unsigned>(ch.share) ? left : ch.share, step = i / mine;
    // (the division leaves scalar registers)
    return __builtin_amdgcn_readfirstlane(
        step < static_cast<unsigned>(ch.tiles) ? static_cast<int>(step * ch.chains + first + i - step * mine) : -1);
}

// A map: (factor, addend), the factor held as a decay is (decay_of), except that
// where 1 - a is 0 it is a = 1, so that -0 stays free for a reset.
constexpr float RESET = -0.f;
__device__ __forceinline__ bool resets(float factor) { return __float_as_uint(factor) == 0x80000000u; }
__device__ __forceinline__ float factor_of(float a, float rest) {
    return __float_as_uint(rest) - 1u < 0x3effffffu ? -rest : a;  // 0 < rest < 0.5
}
// what a map makes of a state
template <bool PACKED>
__device__ __forceinline__ float pass(float2 n, float h) {
    const float through = decay_of(n.x) * h + n.y;
    return PACKED && resets(n.x) ? n.y : through;
}
// Maps joined one by one: the product of their factors, and its complement as a
// sum of complements, 1 - a2 a1 = (1 - a1) + (1 - a2) a1: of products of rounded
// factors it would be off by as much as 1 - a is where all are near 1, and by
// the same on every tile that a state passes.  (One sequence, a = 1 - 6e-6 on each
// of 65536 tokens: off by up to 1.5e-3 of its largest value that way, with the
// sum 2.4e-6.)
template <bool PACKED>
struct Joint {
    float a = 1.f, rest = 0.f, u = 0.f;
    // (f, w, v, cut): a factor, its complement, an addend, and whether the map resets
    __device__ __forceinline__ void then(float f, float w, float v, bool cut) {  // after the maps so far
        w = w * a + rest;
        const float h = f * u + v;
        rest = cut ? 1.f : w;
        u = cut ? v : h;
        a = cut ? RESET : a * f;
    }
    __device__ __forceinline__ void behind(float f, float w, float v, bool cut) {  // before the maps so far
        const bool done = PACKED && resets(a);
        w = w * a + rest;
        const float h = a * v + u;
        rest = (done | cut) ? 1.f : w;
        u = done ? u : h;
        a = (done | cut) ? RESET : a * f;
    }
    __device__ __forceinline__ void then(float2 n) { then(decay_of(n.x), rest_of(n.x), n.y, PACKED && resets(n.x)); }
    __device__ __forceinline__ void behind(float2 n) { behind(decay_of(n.x), rest_of(n.x), n.y, PACKED && resets(n.x)); }
    __device__ __forceinline__ float2 map() const { return make_float2(factor_of(a, rest), u); }
};

// The map of a group of tokens, with its factor and the complement apart: the
// top bit of `value` set where the map resets (by itself, so that a decay that is
// no number has no such bit).
__device__ __forceinline__ float with_mark(float value, bool cut) {
    return __uint_as_float((__float_as_uint(value) & 0x7fffffffu) | static_cast<unsigned>(cut) << 31);
}
__device__ __forceinline__ bool has_mark(float value) { return __float_as_int(value) < 0; }

// Word `at` behind uniform ones: (factor, addend) of a map, or (anything, state).
__device__ __forceinline__ void leave(uint64_t *words, unsigned at, float a, float u) {
    unsigned hi = __float_as_uint(u);
    if (hi == 0xffffffffu) hi = 0x7fc00000u;  // a NaN like any other: NOT_YET stays apart
    __hip_atomic_store(words + at, static_cast<uint64_t>(hi) << 32 | __float_as_uint(a), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 word(uint64_t w) {
    return make_float2(__uint_as_float(static_cast<unsigned>(w)), __uint_as_float(static_cast<unsigned>(w >> 32)));
}

// A look at up to 16 words of a chain, first ones of an order (lane: place jc,
// part jp of the words).  All but `w` is the same in all lanes of a wave.
template <int LOOK>
struct Look {
    uint64_t *words;
    int n, first;  // words wanted, the lane's first
    uint64_t w[LOOK];
    __device__ __forceinline__ bool want(int k) const { return first + k < n; }
    // A first look, long before the words are needed.  No branch around its
    // loads, so that the loads behind them need not be waited for with them:
    // where there are no words it reads zeros.
    __device__ __forceinline__ void start(uint64_t *from, int count, int jc, int jp) {
        words = from;
        n = count;
        first = jp * LOOK;
        const auto b = buffer<uint64_t>(from, 0, n > 0 ? n * CW : 0);
#pragma unroll
        for (int k = 0; k < LOOK; ++k) {
            constexpr int SC1 = 16;  // past the caches that other workgroups' stores do not reach
            w[k] = __builtin_bit_cast(uint64_t, __builtin_amdgcn_raw_buffer_load_b64(b, ((want(k) ? first + k : 0) * CW + jc) * 8, 0, SC1));
        }
    }
    __device__ __forceinline__ void again(int jc) {
        const unsigned at = jc;
#pragma unroll
        for (int k = 0; k < LOOK; ++k)
            if (want(k)) w[k] = __hip_atomic_load(words + (first + k) * CW + at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __device__ __forceinline__ bool there() const {
        int missing = 0;
#pragma unroll
        for (int k = 0; k < LOOK; ++k) missing |= want(k) & (w[k] == NOT_YET);
        return __builtin_amdgcn_ballot_w64(missing != 0) == 0;
    }
    // Waits for the words.  (The first look apart from the loop, which waits for
    // all loads of the wave.)
    __device__ __forceinline__ void wait(const Chain &ch, int jc) {
        if (there()) return;
        unsigned *end = ch.counters + GROUPS * COUNTER_STEP;
        for (int spin = 0; spin < (1 << 18); ++spin) {
            __builtin_amdgcn_s_sleep(1);
            again(jc);
            if (there()) break;
            if ((spin & 255) == 255 &&
                __builtin_amdgcn_readfirstlane(__hip_atomic_load(end, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)))
                break;
            // over a hundred times what a launch takes: the workspace is not this call's alone
            if (spin == (1 << 18) - 1) __hip_atomic_store(end, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    // the words' map
    template <bool PACKED>
    __device__ __forceinline__ float2 map() const {
        Joint<PACKED> m;
#pragma unroll
        for (int k = 0; k < LOOK; ++k) m.then(want(k) ? word(w[k]) : make_float2(1.f, 0.f));
        return m.map();
    }
};

// What tile `step` of a chain looks back at: the maps of its run, the runs of
// its span, and the state before it (of part 0).  The first tile's map holds the
// state that the chain starts from, and no factor: state_out may be state0, and
// what a later tile stores there comes after the first one's read.
template <int LOOK>
struct LookBack {
    Look<LOOK> maps, runs;
    Look<1> state;
    __device__ __forceinline__ void start(const Chain &ch, int64_t chain, int step, int jc, int jp) {
        maps.start(ch.maps + (chain * ch.tiles + step / RUN * RUN) * CW, step % RUN, jc, jp);
        runs.start(ch.runs + (chain * (ch.tiles / RUN) + step / SPAN * (SPAN / RUN)) * CW, step % SPAN / RUN, jc, jp);
        state.start(ch.states + (chain * (ch.tiles / SPAN) + step / SPAN - 1) * CW, jp == 0 && step >= SPAN, jc, 0);
    }
};

// The state that enters tile `step` of a chain (place jc), for all waves; `own`:
// the tile's map, `start`: what the chain starts from, both of wave 0 (jp = 0).
// Leaves the map of a run behind its last tile.  Barriers within.
template <bool PACKED, int PARTS, int LOOK>
__device__ __forceinline__ float enter(const Chain &ch, LookBack<LOOK> &back, int64_t chain, int step, int jc, int jp, float2 own,
                                       float start, float2 (&s_maps)[PARTS][CW], float2 (&s_runs)[PARTS][CW], float (&s_start)[CW]) {
    if (jp == 0 && step + 1 < ch.tiles) {
        if (step == 0) own = make_float2(0.f, pass<PACKED>(own, start));
        leave(back.maps.words, step % RUN * CW + jc, own.x, own.y);
    }
    back.maps.wait(ch, jc);
    s_maps[jp][jc] = back.maps.template map<PACKED>();
    if (jp == 0) s_start[jc] = start;
    __syncthreads();
    if (step >= RUN || step + 1 == RUN) {
        if (jp == 0 && step % RUN == RUN - 1 && step + 1 < ch.tiles) {
            Joint<PACKED> m;
#pragma unroll
            for (int i = 0; i < PARTS; ++i) m.then(s_maps[i][jc]);
            m.then(own);
            const float2 run = m.map();
            leave(back.runs.words, step % SPAN / RUN * CW + jc, run.x, run.y);
        }
        back.runs.wait(ch, jc);
        s_runs[jp][anew(jc)] = back.runs.template map<PACKED>();
        if (jp == 0 && step >= SPAN) {
            back.state.wait(ch, jc);
            s_start[jc] = word(back.state.w[0]).y;
        }
        __syncthreads();
    }
    float h = s_start[jc];
    if (step >= RUN)
#pragma unroll
        for (int i = 0; i < PARTS; ++i) h = pass<PACKED>(s_runs[i][jc], h);
#pragma unroll
    for (int i = 0; i < PARTS; ++i) h = pass<PACKED>(s_maps[i][jc], h);
    return h;
}
__device__ __forceinline__ void leave_state(const Chain &ch, int64_t chain, int step, int jc, float h) {
    if (step % SPAN == SPAN - 1 && step + 1 < ch.tiles) leave(ch.states + (chain * (ch.tiles / SPAN) + step / SPAN) * CW, jc, 0.f, h);
}

// No lane of the kernels branches by itself: what a lane does not need goes to
// NOWHERE, and branches are those of whole waves.  (Where registers are short the
// compiler has moved live values away behind a branch of some lanes before it
// turned the others back on, and they lost theirs.)

// An offset, or nowhere.  (By its top bit, which no offset has: of a ?: the
// compiler makes a branch where it is used more than once.)
__device__ __forceinline__ unsigned only(bool on, unsigned at) { return at | static_cast<unsigned>(!on) << 31; }
static_assert(NOWHERE == 1u << 31, "nowhere is a bit");

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
    __device__ __forceinline__ void load(const int *seq, int64_t row, int r0, int rows) {
        if constexpr (PACKED) {
            const auto b = buffer<int>(seq, row, rows + 2);
#pragma unroll
            for (int k = 0; k < K + 2; ++k) sq[k] = __builtin_amdgcn_raw_buffer_load_b32(b, (r0 + k) * 4, 0, 0);
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k) sq[k + 1] = r0 + k < rows;
        }
    }
    // whether some lane of the wave has a sequence's first or last token
    __device__ __forceinline__ bool edges() const {
        bool edge = false;
#pragma unroll
        for (int k = 0; k < K; ++k) edge = edge | first(k) | last(k);
        return __builtin_amdgcn_ballot_w64(edge) != 0;
    }
    __device__ __forceinline__ bool live(int k) const { return sq[k + 1] != 0; }
    __device__ __forceinline__ bool first(int k) const { return PACKED & live(k) & (sq[k] != sq[k + 1]); }
    __device__ __forceinline__ bool last(int k) const { return PACKED & live(k) & (sq[k + 2] != sq[k + 1]); }
    // offset of the row's sequence in states [N, D] for a channel's byte offset, or nowhere
    // (of no sequence: -4 D, which stays below 2^32 with a vector added)
    __device__ __forceinline__ unsigned state(int k, bool on, unsigned D, unsigned c4) const {
        return only(on, static_cast<unsigned>(sq[k + 1] - 1) * (D * 4) + c4);
    }
};

}  // namespace
}  // namespace scan
}  // namespace gdn2
