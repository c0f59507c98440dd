// linear_chunk.hip -- linear attention with a decay for each head: the
// chunked forward and backward, batched or packed sequences.
//
// Per (sequence, head), with a state S (dk x dv):
//   S_t = a_t S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,   a_t = exp(la_t).
// Over a chunk of C tokens, with g the running sum of la inside the chunk and
// S the state that enters it,
//   o_i = scale (e^{g_i} S^T q_i + sum_{j<=i} e^{g_i-g_j} (q_i . k_j) v_j)
//   S  <- e^{g_C} S + sum_j e^{g_C-g_j} k_j v_j^T.
// Every exponent is a sum of decays over a forward range, so none is
// positive and nothing has to be rescaled.
//
// All three gradients are the same computation on other tensors:
//   dq_t = scale S_t dO_t           = the forward of (dO, v, k), state S^T;
//   dv_t = dS_t^T k_t, dk_t = dS_t v_t, dS_t = a_{t+1} dS_{t+1} + scale q_t dO_t^T
//                                   = the forward of (k, q, dO) and (v, dO, q)
//                                     over the tokens in reverse order, where
//                                     token t carries the decay of token t+1.
// So one kernel, the sweep over rows (x, y, z) = (query, key, value) roles,
// serves the forward and the backward.  The decay's gradient follows from
//   d la_t = <S_e, dS_e> + sum_{t<=i<=e} (q_i . dq_i - k_i . dk_i)
// for any e >= t of the sequence.  The part of each product that a pair of
// tokens in one chunk adds is in both terms, so it is formed once, in the
// sweep of dq, and summed over the chunk alone; the rest, what the state adds,
// is stored per token by the sweeps of dq and dk in fp32, and summed in 64
// bits over a segment from the <S, dS> of its end.
//
// Bound by HBM (the forward reads q, k, v and writes o: 4 dk dv operations
// for 2 (2 dk + 2 dv) bytes a token and head, a quarter of what a large
// product reaches).  Measured, H=16, d=128, bf16, decays and an initial state,
// whole calls in a warm loop: 8 x 4096 tokens 200-212 us (2.7 TB/s; a large
// copy takes 113), 65536 tokens 395-409 us (k and v read twice: 4.0 TB/s), the
// backward of 4 x 4096 tokens 370-400 us.
//
// Long sequences are cut into segments: a state-only sweep forms what every
// segment adds to the state, a scan over the segments turns these into the
// state that enters each, and the sweeps then run over all segments at once.
#include <initializer_list>

#include "chunk_walk.h"
#include "kernels.h"
#include "linear.h"

namespace gdn2 {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr double LOG2E = 1.4426950408889634;
constexpr float LA_MIN = -1e4f;  // exp of anything below is 0 in fp32; keeps differences of sums finite

struct SweepArgs {
    const void *x, *y, *z;   // rows [token, H, dx], [token, H, dx], [token, H, dz]
    void *out;               // rows [token, H, dz]
    const void *w;           // rows [token, H, dz], for u
    float *u, *m;            // [H][tokens]: per token what it adds to the decay's gradient (OUTU, OUTM)
    const float *la;
    const float *s_in;       // [segment][H][dk*dv] or nullptr (zeros)
    float *s_out;            // the same, or nullptr
    double *tot;             // [segment][H]: sum of log2 decays (state-only), or nullptr
    const int32_t *cu;       // packed sequences, one segment each (tab == nullptr)
    const int2 *tab;         // packed sequences cut into segments: first token, end of the sequence
    const int *nsegs;        // number of segments of a packed plan (device), or nullptr
    int64_t T, tokens;       // tokens of a sequence (cu: of the axis), all tokens
    int64_t segs;            // segments launched
    int H, dx, dz;
    int nseg, L;             // segments of a batched sequence, tokens of a segment
    int ncb;                 // column blocks
    int la_tok, rev;
    int s_t;                 // state stored [dz][dx] (the sweep's state is the transpose)
    int gx, gz;              // bytes of one access to x and y rows, to z, w and out rows: 16, 4 or 2
    float p_scale, u_scale, s_scale;
};

struct Seg {
    int64_t lo, hi, end;  // tokens [lo, hi) of a sequence that ends at `end`
};

__device__ __forceinline__ Seg segment(const SweepArgs &a, int64_t seg) {
    Seg r;
    if (a.tab) {
        const int2 e = a.tab[seg];
        r.lo = e.x;
        r.end = e.y;
        r.hi = min(r.lo + a.L, r.end);
    } else if (a.cu) {
        r.lo = min(max(static_cast<int64_t>(a.cu[seg]), int64_t(0)), a.T);
        r.hi = r.end = min(max(static_cast<int64_t>(a.cu[seg + 1]), r.lo), a.T);
    } else {
        const int64_t b = seg / a.nseg, s = seg - b * a.nseg;
        r.lo = b * a.T + s * a.L;
        r.end = (b + 1) * a.T;
        r.hi = min(r.lo + a.L, r.end);
    }
    return r;
}

// Element types.  A fragment holds the 8 contraction slots of one lane for a
// block of 32: lane group lane/16 holds slots 8 (lane/16) .. + 7, lane % 16 is
// the other index.  The slots of a block may be in any order as long as both
// operands use the same one.
template <class T>
struct Elem;

template <>
struct Elem<__bf16> {
    using Frag = bf16x8;
    static constexpr int CT = 64;  // tokens of a chunk
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    // x = p[0] + p[1] + .. with n parts: each part takes the next 8 bits
    template <int N>
    static __device__ __forceinline__ void split(const float (&x)[8], Frag (&p)[N]) {
        float r[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = x[e];
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const f32x2 v = {r[e], r[e + 1]};
                const bf16x2 h = __builtin_convertvector(v, bf16x2);
                p[i][e] = h[0];
                p[i][e + 1] = h[1];
                if (i + 1 < N) {
                    r[e] -= static_cast<float>(h[0]);
                    r[e + 1] -= static_cast<float>(h[1]);
                }
            }
        }
    }
    static __device__ __forceinline__ float at(const Frag &f, int e) { return static_cast<float>(f[e]); }
};

template <>
struct Elem<float> {
    using Frag = f32x8;
    static constexpr int CT = 32;
    static __device__ __forceinline__ f32x4 mma(const Frag &a, const Frag &b, f32x4 c) {
#pragma unroll
        for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
        return c;
    }
    template <int N>
    static __device__ __forceinline__ void split(const float (&x)[8], Frag (&p)[N]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[0][e] = x[e];
    }
    static __device__ __forceinline__ float at(const Frag &f, int e) { return f[e]; }
};

// A row-major LDS tile of COLS columns.  bf16 rows are 16-byte units permuted
// by the row (no padding), so that the 16 rows of a row fragment fall in 16
// different units; a transposed read then takes its banks twice.  fp32 rows
// are padded by 16 bytes.
template <class T, int COLS>
struct Tile;

template <int COLS>
struct Tile<__bf16, COLS> {
    static_assert(COLS == 64 || COLS == 128, "8 or 16 units a row");
    static constexpr int UNITS = COLS / 8, PER = 8, BYTES = COLS * 2;  // PER: elements of a unit
    static __device__ __forceinline__ int unit(int row, int c) {  // byte offset of unit c of a row
        const int f = UNITS == 16 ? ((row & 1) << 2) | ((row >> 1) & 3) | (row & 8) : (row >> 1) & 7;
        return row * BYTES + ((c ^ f) << 4);
    }
    // 8 consecutive columns 8c .. of a row
    static __device__ __forceinline__ bf16x8 row_frag(const char *t, int row, int c) {
        return *reinterpret_cast<const bf16x8 *>(t + unit(row, c));
    }
    // Tokens 32 kt + 8g + e (e = 0..7) of the column that slot lane%16 of a
    // 16-slot tile stands for: slots 4p .. 4p+3 are the 4 columns at half
    // `half` of unit `un`, both given for p = lane%4.  The transposing LDS
    // read gives lane i, element j of 16 lanes what lane 4j + i/4 addresses,
    // element i%4.
    static __device__ __forceinline__ bf16x8 col_frag(const char *t, int kt, int un, int half, int lane) {
        const int row = 8 * (lane >> 4) + ((lane & 15) >> 2);
        typedef __attribute__((address_space(3))) s16x4 lds4;
        const char *p0 = t + 32 * kt * BYTES + unit(row, un) + 8 * half;
        const char *p1 = t + 32 * kt * BYTES + unit(row + 4, un) + 8 * half;
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)p0);
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)p1);
        const s16x8 r = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_bit_cast(bf16x8, r);
    }
    // the 4 columns 4c .. of a row
    static __device__ __forceinline__ f32x4 quad(const char *t, int row, int c) {
        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
        return __builtin_convertvector(*reinterpret_cast<const bf16x4 *>(t + unit(row, c >> 1) + 8 * (c & 1)), f32x4);
    }
};

template <int COLS>
struct Tile<float, COLS> {
    static constexpr int UNITS = COLS / 4, PER = 4, BYTES = COLS * 4 + 16;
    static __device__ __forceinline__ int unit(int row, int c) { return row * BYTES + (c << 4); }
    static __device__ __forceinline__ f32x8 row_frag(const char *t, int row, int c) {
        const f32x4 a = *reinterpret_cast<const f32x4 *>(t + row * BYTES + 32 * c);
        const f32x4 b = *reinterpret_cast<const f32x4 *>(t + row * BYTES + 32 * c + 16);
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    // `un`, `half` as in the bf16 form: given for group lane%4, where the
    // column read here is one of group (lane%16)/4
    static __device__ __forceinline__ f32x8 col_frag(const char *t, int kt, int un, int half, int lane) {
        const int s = lane & 15;
        return column(t, kt, 8 * (un - (lane & 3) + (s >> 2)) + 4 * half + (s & 3), lane);
    }
    static __device__ __forceinline__ f32x8 column(const char *t, int kt, int col, int lane) {
        const float *p = reinterpret_cast<const float *>(t + (32 * kt + 8 * (lane >> 4)) * BYTES) + col;
        f32x8 r;
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = p[e * (BYTES / 4)];
        return r;
    }
    static __device__ __forceinline__ f32x4 quad(const char *t, int row, int c) {
        return *reinterpret_cast<const f32x4 *>(t + unit(row, c));
    }
};

// The score matrix: blocks of 32 columns (tokens j), block kt with the rows
// i >= 32 kt, each row 32 elements.
template <class T>
struct Scores;

template <>
struct Scores<__bf16> {
    static constexpr int ROW = 64, BYTES = (64 + 32) * ROW;
    static __device__ __forceinline__ int at(int kt, int row, int c) {  // unit c (8 columns) of a row of block kt
        return kt * (32 * ROW) + row * ROW + ((c ^ ((row >> 2) & 3)) << 4);
    }
    static __device__ __forceinline__ bf16x8 frag(const char *p, int kt, int row, int g) {
        return *reinterpret_cast<const bf16x8 *>(p + at(kt, row, g));
    }
};

template <>
struct Scores<float> {
    static constexpr int ROW = 32 * 4 + 16, BYTES = 32 * ROW;
    static __device__ __forceinline__ int at(int, int row, int c) { return row * ROW + (c << 4); }  // 4 columns
    static __device__ __forceinline__ f32x8 frag(const char *p, int, int row, int g) {
        const f32x4 a = *reinterpret_cast<const f32x4 *>(p + row * ROW + 32 * g);
        const f32x4 b = *reinterpret_cast<const f32x4 *>(p + row * ROW + 32 * g + 16);
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

// Buffer accesses: a uniform base, a 32-bit lane offset and a uniform one,
// where an offset of NOWHERE reads zeros and stores nothing.
constexpr int NOWHERE = -1;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void *p, int bytes = 0x7fffffff) {
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u >> 32));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>((static_cast<uint64_t>(hi) << 32) | lo), 0, bytes, 0x00027000);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t b, int off, int add) {
    return __builtin_amdgcn_raw_buffer_load_b128(b, off, add, 0);
}
__device__ __forceinline__ float load4(__amdgpu_buffer_rsrc_t b, int off, int add) {
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, off, add, 0));
}
__device__ __forceinline__ void store4(float v, __amdgpu_buffer_rsrc_t b, int off, int add) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), b, off, add, 0);
}

__device__ __forceinline__ bool inside(int p, int len) { return static_cast<unsigned>(p) < static_cast<unsigned>(len); }

// Rows of one tensor for the chunks of a segment, staged in registers: CT
// rows of COLS columns, thread by thread in 16-byte units.  Positions run
// forward from token `first`, or (rev) back from it.
template <class T, int COLS, int CT, int NTH, bool VEC>
struct Stage {
    using Tl = Tile<T, COLS>;
    static constexpr int RX = NTH / Tl::UNITS, N = CT / RX;  // rows of a pass, passes
    static_assert(RX <= CT && CT % RX == 0, "whole passes");
    u32x4 r[N];
    const T *base;  // row of position 0 (rev: of position -(CT-1)), column 0 of the head
    int64_t row;    // elements from one position to the next
    int off;        // this thread's bytes in pass 0 (rev: in the last)
    int add0, step; // bytes of pass 0, from pass to pass
    int r0, c, d, gran;

    __device__ __forceinline__ void init(const void *p, int64_t first, int H, int h, int d_, int col0, bool rev, int gran_, int tid) {
        d = d_;
        gran = gran_;
        const int pitch = H * d;
        row = rev ? -static_cast<int64_t>(pitch) : pitch;
        base = static_cast<const T *>(p) + (first * H + h) * d;
        r0 = tid / Tl::UNITS;
        c = col0 + (tid % Tl::UNITS) * Tl::PER;
        if (rev) base -= static_cast<int64_t>(CT - 1) * pitch;
        off = c < d ? ((rev ? RX - 1 - r0 : r0) * pitch + c) * static_cast<int>(sizeof(T)) : NOWHERE;
        step = (rev ? -RX : RX) * pitch * static_cast<int>(sizeof(T));
        add0 = rev ? -(N - 1) * step : 0;
    }
    // positions p0 .. p0+CT-1, of which [0, len) exist
    __device__ __forceinline__ void load(int p0, int len) {
        const auto b = buffer(base + p0 * row);
        if (VEC || gran == 16) {
#pragma unroll
            for (int i = 0; i < N; ++i) r[i] = load16(b, inside(p0 + r0 + i * RX, len) ? off : NOWHERE, add0 + i * step);
        } else if (gran == 4) {
            constexpr int PER4 = 4 / sizeof(T);
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    r[i][k] = __builtin_amdgcn_raw_buffer_load_b32(
                        b, inside(p0 + r0 + i * RX, len) && c + k * PER4 < d ? off + 4 * k : NOWHERE, add0 + i * step, 0);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                uint32_t e[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    e[k] = __builtin_amdgcn_raw_buffer_load_b16(
                        b, inside(p0 + r0 + i * RX, len) && c + k < d ? off + 2 * k : NOWHERE, add0 + i * step, 0);
#pragma unroll
                for (int k = 0; k < 4; ++k) r[i][k] = (e[2 * k] & 0xffffu) | (e[2 * k + 1] << 16);
            }
        }
    }
    __device__ __forceinline__ void store(char *t, int tid) const {
#pragma unroll
        for (int i = 0; i < N; ++i) *reinterpret_cast<u32x4 *>(t + Tl::unit(r0 + i * RX, tid % Tl::UNITS)) = r[i];
    }
};

// Sum of v over this lane and the lower lanes of the wave, in 64 bits.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, ROWS, 0xf, false);
    return v + __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
__device__ __forceinline__ double wave_prefix(double v) {
    v = dpp_add<0x111, 0xf>(v);  // one, two, four, eight lanes up within rows of 16
    v = dpp_add<0x112, 0xf>(v);
    v = dpp_add<0x114, 0xf>(v);
    v = dpp_add<0x118, 0xf>(v);
    v = dpp_add<0x142, 0xa>(v);  // a row's last lane to the next row
    return dpp_add<0x143, 0xc>(v);  // the lower half's last lane to the upper half
}
__device__ __forceinline__ double last_lane(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(u), 63), hi = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), 63);
    return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
// Sum over the 16 lanes of a row, in its last lane.
__device__ __forceinline__ float row16_sum(float v) {
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x111, 0xf, 0xf, false));
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x112, 0xf, 0xf, false));
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x114, 0xf, 0xf, false));
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x118, 0xf, 0xf, false));
    return v;
}

// Sum over 4 or 8 neighbouring lanes, on each of them.
template <int N>
__device__ __forceinline__ float lanes_sum(float v) {
    static_assert(N == 4 || N == 8, "lanes of a half row");
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xb1, 0xf, 0xf, false));  // lane ^ 1
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x4e, 0xf, 0xf, false));  // lane ^ 2
    if (N == 8)  // the mirrored lane of eight, in the other four
        v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x141, 0xf, 0xf, false));
    return v;
}

// What a sweep does: its output parts.
constexpr int STATE = 0;  // the state only
constexpr int OUT = 1;    // outputs (and the state)
constexpr int OUTU = 2;   // outputs and u, the read's row products <w, x S>
constexpr int OUTM = 3;   // OUTU, and in u what the pairs inside a chunk add

template <class T, int DX, int NC, int NT, int KSP>
struct Shape {
    static constexpr int CT = Elem<T>::CT, NW = NC * KSP, WC = NC * 16 * NT;  // columns of a workgroup
    using TX = Tile<T, DX>;
    using TZ = Tile<T, WC>;
    static constexpr int XB = CT * TX::BYTES, ZB = CT * TZ::BYTES;
    static constexpr int OB = KSP > 1 ? NW * (CT / 32) * NT * 1024 : 0;  // read sums passed between waves
    static constexpr size_t bytes(int mode, int np) {
        return CT * 8 + 2 * CT * 4 + 16 + (mode == STATE ? 1 : 2) * XB + (mode >= OUTU ? 2 : 1) * ZB +
               (mode == STATE ? 0 : np * Scores<T>::BYTES + OB) + (mode >= OUTU ? NW * CT * 16 : 0) +
               (mode == OUTM ? (CT / 16 + 1) * CT * 16 : 0);
    }
};

// One workgroup of NW waves: one segment of one head, WC columns of z.  A
// wave holds DX x 16 NT of the state in accumulators for the whole segment:
// tile (m, t), m = 2 ks + hf: row slot s = 4p + r is channel 32 ks + 8p + 4hf + r
// and column slot s = 4p + r is column 8p + 4t + r of the wave's (NT = 2), so
// that 8 contraction slots of a lane are 8 neighbouring channels, and a lane's
// outputs 8 neighbouring columns.
//
// The operands made here are rounded to bf16 parts: the score matrix to NP of
// them, the state to NS, the decayed values that update the state to NU (three
// parts hold all 24 bits; fp32 inputs are not split).  Where only bf16 results
// follow, two parts: they leave 2^-16 of an operand, where the result's own
// rounding leaves 2^-8.  Against fp64, o and dv are then as far off as fp32
// sums rounded once (relative 1.66e-3; with the state in one part up to
// 2.25e-3 where it dominates).  Three parts everywhere give the same 1.66e-3
// and take 234 us for 207 (8 x 4096 tokens, H=16, d=128) and 555 for 409
// (65536 tokens).
//
// OUTU and OUTM (all of z's columns in one workgroup): per token what it adds
// to the decay's gradient, through the state and (OUTM) inside its chunk,
//   u_i = <w_i, e^{g_i} S^T x_i>,   m_i = sum_{j<i} M_ij - sum_{j>i} M_ji,
//   M_ij = (score i, j) (w_i . z_j):
// a pair inside a chunk enters both its ends with the same fp32 value, so the
// sum of m over a chunk's tail keeps its precision.
template <class T, int DX, int NCW, int NT, int KSP, int MODE, int NP, int NS, int NU, bool VEC>
__device__ __forceinline__ void sweep_body(const SweepArgs &a, int64_t item, char *smem) {
    using E = Elem<T>;
    using Frag = typename E::Frag;
    using Sh = Shape<T, DX, NCW, NT, KSP>;
    using TX = typename Sh::TX;
    using TZ = typename Sh::TZ;
    using Sc = Scores<T>;
    constexpr int CT = E::CT, NW = Sh::NW, NTH = 64 * NW, ESZ = sizeof(T);
    constexpr int KT = CT / 32, RT = CT / 16, KS = DX / 32;     // blocks of tokens, row tiles, blocks of channels
    constexpr int KSW = KS / KSP, MT = 2 * KSW, RTW = RT / KSP;  // a wave's blocks, state tiles, row tiles

    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, ls = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kp = KSP > 1 ? wave / NCW : 0, cw = KSP > 1 ? wave % NCW : wave;  // the wave's channels and columns
    const int ch0 = 32 * KSW * kp;
    const int cb = static_cast<int>(item % a.ncb);
    const int64_t sh = item / a.ncb;  // segment * H + head
    const int64_t seg = sh / a.H;
    const int h = static_cast<int>(sh - seg * a.H);
    if (a.nsegs && seg >= *a.nsegs) return;
    const Seg sg = segment(a, seg);
    const int len = __builtin_amdgcn_readfirstlane(static_cast<int>(sg.hi - sg.lo));
    const int col0 = cb * Sh::WC, wcol = 16 * NT * cw;  // first column of the workgroup, of the wave in it
    const bool rev = a.rev;
    const int64_t first = rev ? sg.hi - 1 : sg.lo;  // token of position 0

    double *s_g = reinterpret_cast<double *>(smem);
    float *s_e = reinterpret_cast<float *>(s_g + CT);  // s_scale e^{g_i}
    float *s_f = s_e + CT;                              // u_scale e^{g_C - g_j}
    float *s_gam = s_f + CT;
    char *s_y = reinterpret_cast<char *>(s_gam + 4);
    char *s_z = s_y + Sh::XB;
    char *s_x = s_z + Sh::ZB;
    char *s_p = s_x + Sh::XB;
    char *s_w = s_p + NP * Sc::BYTES;
    float *s_u = reinterpret_cast<float *>(s_w + Sh::ZB);  // [NW][CT][4 lane groups]
    // [CT/16 blocks][CT/16 + 1][4][16]: sums of the block's tiles over their
    // rows' four lane groups, then over their columns (one of the four)
    float *s_m = s_u + (MODE >= OUTU ? 4 * NW * CT : 0);
    // [NW][RTW][NT][64 lanes][4]
    float *s_o = MODE >= OUTU ? s_m + (MODE == OUTM ? 4 * (RT + 1) * CT : 0) : reinterpret_cast<float *>(s_w);

    // column of slot s of tile t, relative to the wave's
    auto zcol = [](int t, int s) { return NT == 2 ? 8 * (s >> 2) + 4 * t + (s & 3) : s; };

    // the state's elements of this lane: channels 32 ks + 4 hf + 8g + r
    f32x4 S[MT][NT];
    const int dkv = a.dx * a.dz;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) S[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const bool all_ch = a.dx == DX;
    // fp32: blocks of 32 channels that the rows do not have are passed over
    const int live_ch = __builtin_amdgcn_readfirstlane(a.dx);
    auto past = [&](int ch) { return ESZ == 4 && ch >= live_ch; };
    int soff[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int col = col0 + wcol + zcol(t, ls);
        soff[t] = col < a.dz ? 4 * ((ch0 + 8 * g) * a.dz + col) : NOWHERE;
    }
    if (MODE != STATE && a.s_in) {
        const auto b = buffer(a.s_in + sh * dkv, 4 * dkv);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int ch = 32 * (m >> 1) + 4 * (m & 1);
                if (!a.s_t) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        S[m][t][r] = load4(b, all_ch || ch0 + ch + 8 * g + r < a.dx ? soff[t] : NOWHERE, 4 * (ch + r) * a.dz);
                } else {
                    const int col = col0 + wcol + zcol(t, ls);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int c = ch0 + ch + 8 * g + r;
                        S[m][t][r] = load4(b, c < a.dx && col < a.dz ? 4 * (col * a.dx + c) : NOWHERE, 0);
                    }
                }
            }
    }
    // the state is waited for here: a wait inside the chunk loop would also
    // wait for the next chunk's rows
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) asm volatile("" : "+v"(S[m][t]));
    if (MODE != STATE)  // the score tiles above the diagonal stay zero
        for (int i = tid; i < NP * Sc::BYTES / 4; i += NTH) reinterpret_cast<uint32_t *>(s_p)[i] = 0;

    Stage<T, DX, CT, NTH, VEC> sx, sy;
    Stage<T, Sh::WC, CT, NTH, VEC> sz, sw;
    sy.init(a.y, first, a.H, h, a.dx, 0, rev, a.gx, tid);
    sz.init(a.z, first, a.H, h, a.dz, col0, rev, a.gz, tid);
    if (MODE != STATE) sx.init(a.x, first, a.H, h, a.dx, 0, rev, a.gx, tid);
    if (MODE >= OUTU) sw.init(a.w, first, a.H, h, a.dz, col0, rev, a.gz, tid);
    double total = 0.0;  // log2 decays of the staged chunks (last wave)
    float la_next = 0.f;
    // position p takes the decay of token first + p, or (rev) first - p + 1,
    // the token behind it: none for the sequence's last token
    const int64_t la_pitch = a.la_tok ? a.H : 0, la_row = rev ? -la_pitch : la_pitch;
    const float *la_base = a.la + h + (rev ? first + 1 - (CT - 1) : first) * la_pitch;
    const int la_off = static_cast<int>(rev ? CT - 1 - lane : lane) * static_cast<int>(la_pitch) * 4;
    const int la_skip = rev && sg.hi == sg.end ? -1 : 0;  // position 0 has none
    auto load_first = [&](int p0) {
        sy.load(p0, len);
        if (MODE != STATE) sx.load(p0, len);
    };
    auto load_second = [&](int p0) {
        sz.load(p0, len);
        if (MODE >= OUTU) sw.load(p0, len);
        if (wave == NW - 1)  // the decay of each position
            la_next = load4(buffer(la_base + p0 * la_row), lane < CT && inside(p0 + lane + la_skip, len + la_skip) ? la_off : NOWHERE, 0);
    };
    // the loaded chunk into LDS, its decays summed
    auto stage_chunk = [&] {
        sy.store(s_y, tid);
        sz.store(s_z, tid);
        if (MODE != STATE) sx.store(s_x, tid);
        if (MODE >= OUTU) sw.store(s_w, tid);
        if (wave == NW - 1) {
            // running sums in 64 bits: a far reset must not cost the decays
            // that follow it their low bits
            const double v = wave_prefix(static_cast<double>(la_next < LA_MIN ? LA_MIN : la_next) * LOG2E);
            const double all = last_lane(v);
            if (lane < CT) {
                s_g[lane] = v;
                s_e[lane] = a.s_scale * __builtin_amdgcn_exp2f(static_cast<float>(v));
                s_f[lane] = a.u_scale * __builtin_amdgcn_exp2f(static_cast<float>(all - v));
            }
            if (lane == 0) *s_gam = __builtin_amdgcn_exp2f(static_cast<float>(all));
            total += all;
        }
    };
    // this lane's outputs: NC neighbouring columns of token row 16 rt + ls
    constexpr int NC = 4 * NT;
    const int oc = col0 + wcol + NC * g;
    const int64_t orow = static_cast<int64_t>(a.H) * a.dz;
    T *obase = MODE != STATE ? static_cast<T *>(a.out) + (first * a.H + h) * a.dz : nullptr;
    const int ooff = oc < a.dz ? ((rev ? 15 - ls : ls) * static_cast<int>(orow) + oc) * ESZ : NOWHERE;

    // chunks keep the forward order's borders: in reverse the ragged one is first
    const int begin = rev ? -((CT - len % CT) % CT) : 0;
    if (len > 0) {
        load_first(begin);
        load_second(begin);
        stage_chunk();
    }
    __syncthreads();

    for (int p0 = begin; len > 0; p0 += CT) {
        // the next chunk's loads, in two parts: a CU takes 64 bytes a cycle
        const bool more = chunk_follows(p0, len, CT);
        if (more) load_first(p0 + CT);
        if (MODE == STATE && more) load_second(p0 + CT);

        Frag zf[KT][NT];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if constexpr (NT == 2)
                    zf[kt][t] = TZ::col_frag(s_z, kt, (wcol >> 3) + (lane & 3), t, lane);
                else if constexpr (ESZ == 2)
                    zf[kt][t] = TZ::col_frag(s_z, kt, (wcol >> 3) + ((lane >> 1) & 1), lane & 1, lane);
                else
                    zf[kt][t] = TZ::column(s_z, kt, wcol + ls, lane);
            }

        f32x4 O[RT][NT];
        if constexpr (MODE != STATE) {
            // scores, transposed (rows j, columns i), so that a lane holds
            // four neighbouring j of one i; 16 x 16 tiles on and below the diagonal
            // Surplus waves form the last tile again and write the same values.
            constexpr int TILES = RT * (RT + 1) / 2, MINE = (TILES + NW - 1) / NW;
            auto product = [&](int it, int jt) {
                f32x4 sc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    if (past(32 * ks)) break;
                    sc = E::mma(TX::row_frag(s_y + 16 * jt * TX::BYTES, ls, 4 * ks + g),
                                TX::row_frag(s_x + 16 * it * TX::BYTES, ls, 4 * ks + g), sc);
                }
                return sc;
            };
            auto pairs = [&](int it, int jt) {  // w_i . z_j
                f32x4 m = {0.f, 0.f, 0.f, 0.f};
                if constexpr (MODE == OUTM)
#pragma unroll
                    for (int ks = 0; ks < Sh::WC / 32; ++ks)
                        m = E::mma(TZ::row_frag(s_z + 16 * jt * TZ::BYTES, ls, 4 * ks + g),
                                   TZ::row_frag(s_w + 16 * it * TZ::BYTES, ls, 4 * ks + g), m);
                return m;
            };
            auto finish = [&](int it, int jt, f32x4 sc, f32x4 m) {
                const int i = 16 * it + ls, j = 16 * jt + 4 * g;
                const double gi = s_g[i];
                f32x4 pr;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float d = a.p_scale * __builtin_amdgcn_exp2f(static_cast<float>(gi - s_g[j + r]));
                    float v = sc[r] * d;
                    asm("" : "+v"(v));  // formed on every lane: a branch costs more
                    pr[r] = j + r <= i ? v : 0.f;
                }
                if constexpr (ESZ == 2) {
                    f32x4 rest = pr;
                    const int at = Sc::at(jt >> 1, i, 2 * (jt & 1) + (g >> 1)) + 8 * (g & 1);
#pragma unroll
                    for (int q = 0; q < NP; ++q) {
                        const bf16x2 lo = __builtin_convertvector((f32x2{rest[0], rest[1]}), bf16x2);
                        const bf16x2 hi = __builtin_convertvector((f32x2{rest[2], rest[3]}), bf16x2);
                        const uint2 w = {__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
                        *reinterpret_cast<uint2 *>(s_p + q * Sc::BYTES + at) = w;
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            rest[r] -= static_cast<float>(lo[r]);
                            rest[2 + r] -= static_cast<float>(hi[r]);
                        }
                    }
                } else {
                    *reinterpret_cast<f32x4 *>(s_p + Sc::at(0, i, j >> 2)) = pr;
                }
                if constexpr (MODE == OUTM) {
                    float rs = 0.f;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        m[r] = j + r < i ? m[r] * pr[r] : 0.f;
                        rs += m[r];
                        m[r] = row16_sum(m[r]);
                    }
                    s_m[((it * (RT + 1) + jt) * 4 + g) * 16 + ls] = rs;
                    if (ls == 15) *reinterpret_cast<f32x4 *>(s_m + (jt * (RT + 1) + it + 1) * 64 + 4 * g) = m;
                }
            };
            auto tile_i = [&](int n) { return static_cast<int>((0x3333222110ull >> (4 * n)) & 15); };
            auto tile_j = [&](int n) { return static_cast<int>((0x3210210100ull >> (4 * n)) & 15); };
            if constexpr (NW == 8) {  // one workgroup a CU: all at once, branch-free
                f32x4 sc[MINE], m[MINE];
                int n[MINE];
#pragma unroll
                for (int u = 0; u < MINE; ++u) {
                    n[u] = min(wave + u * NW, TILES - 1);
                    sc[u] = product(tile_i(n[u]), tile_j(n[u]));
                    m[u] = pairs(tile_i(n[u]), tile_j(n[u]));
                }
#pragma unroll
                for (int u = 0; u < MINE; ++u) finish(tile_i(n[u]), tile_j(n[u]), sc[u], m[u]);
            } else {  // two: one by one, in fewer registers
#pragma unroll 1
                for (int n = wave; n < TILES; n += NW) finish(tile_i(n), tile_j(n), product(tile_i(n), tile_j(n)), pairs(tile_i(n), tile_j(n)));
            }

            if (more) load_second(p0 + CT);

            // outputs, transposed: x S first, which needs no scores
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int t = 0; t < NT; ++t) O[rt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
            if constexpr (MODE >= OUTU && NS > 1) {
                // The small parts of all channels first: what a matrix
                // instruction adds is cut to fp32 at the size that the sum has
                // by then.  Here and in the state's update it takes the error
                // of d_log_decay from 9.1e-7 to 6.5e-7 (4 x 4096 tokens, H=16,
                // d=128), and the products of two row tiles in turn take the
                // whole backward from 377 to 372 us.
                Frag sf[KSW][NT][NS];
#pragma unroll
                for (int ks = 0; ks < KSW; ++ks)
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = S[2 * ks + (e >> 2)][t][e & 3];
                        E::template split<NS>(v, sf[ks][t]);
                    }
#pragma unroll
                for (int rt = 0; rt < RT; rt += 2) {
                    Frag xf[2][KSW];
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int ks = 0; ks < KSW; ++ks)
                            xf[k][ks] = TX::row_frag(s_x + 16 * (rt + k) * TX::BYTES, ls, (ch0 >> 3) + 4 * ks + g);
#pragma unroll
                    for (int q = NS - 1; q >= 0; --q)
#pragma unroll
                        for (int ks = 0; ks < KSW; ++ks)
#pragma unroll
                            for (int t = 0; t < NT; ++t)
#pragma unroll
                                for (int k = 0; k < 2; ++k) O[rt + k][t] = E::mma(sf[ks][t][q], xf[k][ks], O[rt + k][t]);
                }
            } else {
                // One block of channels at a time, its small part first: all
                // channels' parts at once do not fit two workgroups' registers.
#pragma unroll
                for (int ks = 0; ks < KSW; ++ks) {
                    if (past(ch0 + 32 * ks)) break;
                    Frag sf[NT][NS];
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = S[2 * ks + (e >> 2)][t][e & 3];
                        E::template split<NS>(v, sf[t]);
                    }
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        const Frag xf = TX::row_frag(s_x + 16 * rt * TX::BYTES, ls, (ch0 >> 3) + 4 * ks + g);
#pragma unroll
                        for (int q = NS - 1; q >= 0; --q)
#pragma unroll
                            for (int t = 0; t < NT; ++t) O[rt][t] = E::mma(sf[t][q], xf, O[rt][t]);
                    }
                }
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const float e = s_e[16 * rt + ls];
#pragma unroll
                for (int t = 0; t < NT; ++t) O[rt][t] *= e;
                if constexpr (MODE >= OUTU) {
                    float us = 0.f;
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const f32x4 w = TZ::quad(s_w + 16 * rt * TZ::BYTES, ls, (wcol >> 2) + NT * g + t);
#pragma unroll
                        for (int r = 0; r < 4; ++r) us += O[rt][t][r] * w[r];
                    }
                    s_u[(wave * CT + 16 * rt + ls) * 4 + g] = us;
                }
            }
            if constexpr (KSP > 1)  // the other half's row tiles go to the wave that finishes them
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
                    if (rt / RTW != kp)
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            *reinterpret_cast<f32x4 *>(s_o + (((wave * RTW + rt % RTW) * NT + t) * 64 + lane) * 4) = O[rt][t];
        }

        // the state: decayed, plus the chunk's products
        const float gam = *s_gam;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t) S[m][t] *= gam;
        Frag zu[KT][NT][NU];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            const f32x4 f0 = *reinterpret_cast<const f32x4 *>(s_f + 32 * kt + 8 * g);
            const f32x4 f1 = *reinterpret_cast<const f32x4 *>(s_f + 32 * kt + 8 * g + 4);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = (e < 4 ? f0[e & 3] : f1[e & 3]) * E::at(zf[kt][t], e);
                E::template split<NU>(v, zu[kt][t]);
            }
        }
#pragma unroll
        for (int m = 0; m < MT; m += 2) {  // two tiles at a time: independent products between dependent ones
            if (past(ch0 + 16 * m)) break;
            const int un = (ch0 >> 3) + 4 * (m >> 1) + (lane & 3);
            Frag y[KT][2];
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int k = 0; k < 2; ++k) y[kt][k] = TX::col_frag(s_y, kt, un, k, lane);
            // the small parts of all blocks first: a product is cut to fp32 at
            // the size that its sum has by then
#pragma unroll
            for (int q = NU - 1; q >= 0; --q)
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int k = 0; k < 2; ++k) S[m + k][t] = E::mma(y[kt][k], zu[kt][t][q], S[m + k][t]);
        }

        __syncthreads();  // the scores are written, the tiles read
        if (more) stage_chunk();

        if constexpr (MODE != STATE) {
            if constexpr (MODE >= OUTU) {  // NW neighbouring lanes a token
                const int i = tid / NW, part = tid % NW, p = p0 + i;
                float us = 0.f, ms = 0.f;
                if (i < CT) {
                    const f32x4 v = *reinterpret_cast<const f32x4 *>(s_u + (part * CT + i) * 4);
                    us = (v[0] + v[1]) + (v[2] + v[3]);
                    if constexpr (MODE == OUTM) {
                        const int blk = i >> 4;
#pragma unroll
                        for (int q = part; q <= RT; q += NW) {
                            const float *m = s_m + (blk * (RT + 1) + q) * 64 + (i & 15);
                            ms += q <= blk ? (m[0] + m[16]) + (m[32] + m[48]) : -m[0];
                        }
                    }
                }
                us = lanes_sum<NW>(us);
                if constexpr (MODE == OUTM) ms = lanes_sum<NW>(ms);
                if (i < CT && part == 0 && inside(p, len)) {
                    const int64_t at = static_cast<int64_t>(h) * a.tokens + (rev ? first - p : first + p);
                    a.u[at] = us;
                    if constexpr (MODE == OUTM) a.m[at] = ms;
                }
            }
            // a wave finishes RTW row tiles from rt0 on
            const int rt0 = RTW * kp;
            f32x4 R[RTW][NT];
#pragma unroll
            for (int q = 0; q < RTW; ++q)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if constexpr (KSP > 1) {
                        const int other = wave < NCW ? wave + NCW : wave - NCW;
                        R[q][t] = (kp ? O[RTW + q][t] : O[q][t]) +
                                  *reinterpret_cast<const f32x4 *>(s_o + (((other * RTW + q) * NT + t) * 64 + lane) * 4);
                    } else {
                        R[q][t] = O[q][t];
                    }
                }
#pragma unroll
            for (int q = 0; q < RTW; ++q)
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
                    if (KSP > 1 ? (kt == 0 || kp > 0) : 32 * kt <= 16 * q + 15) {
#pragma unroll
                        for (int n = 0; n < NP; ++n) {
                            const Frag pf = Sc::frag(s_p + n * Sc::BYTES + 16 * (rt0 + q) * Sc::ROW, kt, ls, g);
#pragma unroll
                            for (int t = 0; t < NT; ++t) R[q][t] = E::mma(zf[kt][t], pf, R[q][t]);
                        }
                    }
            {
                T *o = obase + (rev ? -(p0 + CT - 1) : p0) * orow;
                const auto b = buffer(o);
#pragma unroll
                for (int q = 0; q < RTW; ++q) {
                    const int p = p0 + 16 * (rt0 + q) + ls;
                    // 16-byte stores with a register as their uniform offset
                    // have written registers that the next instruction
                    // overwrote: the whole offset goes into the lane's
                    const int off = inside(p, len) && ooff != NOWHERE
                                        ? ooff + 16 * (rev ? RT - 1 - rt0 - q : rt0 + q) * static_cast<int>(orow) * ESZ
                                        : NOWHERE;
                    uint32_t w[NC * ESZ / 4];  // the row's outputs of this lane
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int r = 0; r < 4; r += 4 / ESZ) {
                            if constexpr (ESZ == 2)
                                w[2 * t + r / 2] = __builtin_bit_cast(
                                    uint32_t, __builtin_convertvector((f32x2{R[q][t][r], R[q][t][r + 1]}), bf16x2));
                            else
                                w[4 * t + r] = __float_as_uint(R[q][t][r]);
                        }
                    if (VEC || a.gz == 16) {
                        if constexpr (NC * ESZ == 8)
                            __builtin_amdgcn_raw_buffer_store_b64((u32x2{w[0], w[1]}), b, off, 0, 0);
                        else
#pragma unroll
                            for (int k = 0; k < NC * ESZ / 4; k += 4)
                                __builtin_amdgcn_raw_buffer_store_b128((u32x4{w[k], w[k + 1], w[k + 2], w[k + 3]}), b,
                                                                       oc + 4 * k / ESZ < a.dz && off != NOWHERE ? off + 4 * k : NOWHERE, 0, 0);
                    } else if (a.gz == 4) {
#pragma unroll
                        for (int k = 0; k < NC * ESZ / 4; ++k)
                            __builtin_amdgcn_raw_buffer_store_b32(
                                w[k], b, oc + 4 * k / ESZ < a.dz && off != NOWHERE ? off + 4 * k : NOWHERE, 0, 0);
                    } else {
#pragma unroll
                        for (int k = 0; k < NC; ++k)
                            __builtin_amdgcn_raw_buffer_store_b16(
                                static_cast<uint16_t>(w[k / 2] >> (16 * (k & 1))), b,
                                oc + k < a.dz && off != NOWHERE ? off + 2 * k : NOWHERE, 0, 0);
                    }
                }
            }
        }
        if (!more) break;
        __syncthreads();  // the next chunk is staged, the scores read
    }

    if (a.s_out) {  // (in reverse: the first token's decay is the scan's to apply)
        const auto b = buffer(a.s_out + sh * dkv, 4 * dkv);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int ch = 32 * (m >> 1) + 4 * (m & 1) + r;
                    store4(S[m][t][r], b, all_ch || ch0 + ch + 8 * g < a.dx ? soff[t] : NOWHERE, 4 * ch * a.dz);
                }
    }
    if (MODE == STATE && a.tot && cb == 0 && tid == NTH - 64) a.tot[sh] = total;
}

// Workgroups with neighbouring numbers run on different XCDs (eight, in
// turn); the column blocks of one segment share its x and y rows, so they are
// numbered to land on the same one.
__device__ __forceinline__ int64_t xcd_item(int64_t b, int64_t segheads, int ncb) {
    const int64_t xcd = b & 7, q = b >> 3;
    const int64_t sh = (q / ncb) * 8 + xcd;
    return sh < segheads ? sh * ncb + q % ncb : -1;
}
__host__ int64_t xcd_blocks(int64_t segheads, int ncb) { return (segheads + 7) / 8 * 8 * ncb; }

template <class T, int DX, int NCW, int NT, int KSP, int MODE, int NP, int NS, int NU, bool VEC>
__global__ void __launch_bounds__(64 * NCW * KSP, 2) sweep_kernel(SweepArgs a) {
    extern __shared__ __align__(16) char smem[];
    const int64_t item = xcd_item(blockIdx.x, a.segs * a.H, a.ncb);
    if (item < 0) return;
    sweep_body<T, DX, NCW, NT, KSP, MODE, NP, NS, NU, VEC>(a, item, smem);
}

// The two state sweeps of the backward, and its three gradient sweeps, in one
// launch each.  The gradient sweeps go by groups of segments and heads, one
// sweep after the other: most CUs then run the same instructions, and the
// rows come from the caches the second and third time.  (At 256
// segments and heads of 1024 tokens the whole backward takes 372 us; all of one
// sweep first 374, the three of a segment next to each other 398.)
constexpr int SWEEP_GROUP = 128;

struct Sweeps {
    SweepArgs s[3];
};

template <class T, int DX, int NCW, bool VEC>
__global__ void __launch_bounds__(64 * NCW, 2) state_pair_kernel(Sweeps a) {
    extern __shared__ __align__(16) char smem[];
    const int64_t q = blockIdx.x >> 3, sh = (q >> 1) * 8 + (blockIdx.x & 7);
    if (sh >= a.s[0].segs * a.s[0].H) return;
    sweep_body<T, DX, NCW, 1, 1, STATE, 1, 1, sizeof(T) == 2 ? 3 : 1, VEC>(a.s[q & 1], sh, smem);
}

template <class T, int DX, int NCW, bool VEC>
__global__ void __launch_bounds__(64 * NCW, 2) gradient_kernel(Sweeps a) {
    extern __shared__ __align__(16) char smem[];
    constexpr bool B = sizeof(T) == 2;
    const int64_t each = SWEEP_GROUP, in = blockIdx.x % (3 * each), sh = blockIdx.x / (3 * each) * each + in % each;
    if (sh >= a.s[0].segs * a.s[0].H) return;
    switch (in / each) {
        case 0: sweep_body<T, DX, NCW, 1, 1, OUTM, B ? 2 : 1, B ? 3 : 1, B ? 3 : 1, VEC>(a.s[0], sh, smem); break;
        case 1: sweep_body<T, DX, NCW, 1, 1, OUTU, B ? 2 : 1, B ? 3 : 1, B ? 3 : 1, VEC>(a.s[1], sh, smem); break;
        default: sweep_body<T, DX, NCW, 1, 1, OUT, B ? 2 : 1, B ? 2 : 1, B ? 2 : 1, VEC>(a.s[2], sh, smem); break;
    }
}

// The scan over a sequence's segments: what each adds to the state becomes
// the state that enters it, in place.  One lane per state element.
struct ScanArgs {
    float *tab;           // [segment][H][dk*dv]
    const double *tot;    // [segment][H]
    const float *init;    // [N][H][dk*dv] or nullptr
    float *fin;           // [N][H][dk*dv] or nullptr
    const int *pfx;       // packed: segments before each sequence, or nullptr
    const int2 *seq;      // packed: token ranges
    const float *la;
    int64_t N, T;
    int64_t dkv;
    int H, nseg, rev, la_tok;
};

struct Scans {
    ScanArgs s[2];
};

// V elements of the state a lane (V = 4: whole 16-byte units).  One state a
// workgroup of x, its blocks along y: up to 64 of them for 127 x 127 elements,
// which together with 2^20 states would be more lanes than one axis may have.
template <int V>
__global__ void __launch_bounds__(256) segment_scan_kernel(Scans two) {
    constexpr int AHEAD = 8;  // segments whose loads are in flight together
    typedef float Fv __attribute__((ext_vector_type(V)));
    const ScanArgs &a = two.s[blockIdx.z];
    const int64_t sh = blockIdx.x, n = sh / a.H;
    const int h = static_cast<int>(sh - n * a.H);
    const int64_t e = (static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x) * V;
    if (e >= a.dkv) return;
    const int64_t s0 = a.pfx ? a.pfx[n] : n * a.nseg;
    const int cnt = a.pfx ? a.pfx[n + 1] - a.pfx[n] : a.nseg;
    auto at = [&](const float *p) { return reinterpret_cast<const Fv *>(p); };
    Fv cur = 0.f;
    if (a.init)
#pragma unroll
        for (int k = 0; k < V; ++k) cur[k] = a.init[sh * a.dkv + e + k];  // a caller's state: any alignment
    for (int i = 0; i < cnt; i += AHEAD) {
        Fv *p[AHEAD], add[AHEAD];
        float f[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {  // past the last: the last once more, not used
            const int m = min(i + k, cnt - 1);
            const int64_t sl = (s0 + (a.rev ? cnt - 1 - m : m)) * a.H + h;
            p[k] = const_cast<Fv *>(at(a.tab + sl * a.dkv + e));
            add[k] = *p[k];
            f[k] = __builtin_amdgcn_exp2f(static_cast<float>(a.tot[sl]));
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (i + k < cnt) {
                *p[k] = cur;
                cur = cur * f[k] + add[k];
            }
    }
    if (a.fin) {
        const int64_t lo = a.pfx ? a.seq[n].x : n * a.T;
        if (a.rev && cnt > 0) cur *= __expf(a.la[a.la_tok ? lo * a.H + h : h]);
#pragma unroll
        for (int k = 0; k < V; ++k) a.fin[sh * a.dkv + e + k] = cur[k];
    }
}

// d la of a segment: its last token's <S, dS>, then back over the segment what
// its tokens open and close of the state's part, and over each chunk its pairs;
// in 64 bits, a wave on the 64 tokens of a chunk (or two chunks of 32).  One workgroup per (segment, head).
struct DecayArgs {
    const float *uq, *uk, *m;  // [H][tokens]
    const float *s_tab, *d_tab;  // states entering the segments, forward and reverse
    const float *s_fin;     // [N][H][dk*dv] final states
    const float *la;
    float *d_la;            // [token, H] (la_tok)
    double *part;           // [segment][H] sums (per-head decays)
    const int2 *tab, *seq;
    const int *pfx;
    int64_t N, T, tokens, segs, dkv;
    int H, nseg, L, la_tok, half;  // half: chunks of 32 tokens, not 64
};

template <int NTH>
__global__ void __launch_bounds__(NTH) decay_grad_kernel(DecayArgs a) {
    constexpr int NW = NTH / 64;
    __shared__ double red[NW];
    const int64_t sh = blockIdx.x, seg = sh / a.H;
    const int h = static_cast<int>(sh - seg * a.H), tid = threadIdx.x, lane = tid & 63;
    if (a.pfx && seg >= a.pfx[a.N]) return;
    int64_t lo, end, n;
    bool last;
    if (a.tab) {
        const int2 e = a.tab[seg];
        lo = e.x;
        end = e.y;
        last = lo + a.L >= end;
        int l = 0, r = static_cast<int>(a.N) - 1;  // the sequence: the last that starts at or before seg
        while (l < r) {
            const int mid = (l + r + 1) >> 1;
            if (a.pfx[mid] <= seg) l = mid;
            else r = mid - 1;
        }
        n = l;
        last = last || seg + 1 >= a.pfx[a.N];  // offsets that break the rules may cut a sequence short
    } else {
        n = seg / a.nseg;
        lo = n * a.T + (seg - n * a.nseg) * a.L;
        end = (n + 1) * a.T;
        last = seg - n * a.nseg == a.nseg - 1;
    }
    const int64_t hi = min(lo + a.L, end);
    const float *s = last ? a.s_fin + (n * a.H + h) * a.dkv : a.s_tab + (sh + a.H) * a.dkv;
    const float *d = a.d_tab + sh * a.dkv;
    double x = 0.0;
    if (a.dkv % 4 == 0) {
        for (int64_t e = 4 * tid; e < a.dkv; e += 4 * NTH) {
            const float4 p = *reinterpret_cast<const float4 *>(s + e), q = *reinterpret_cast<const float4 *>(d + e);
            x += (static_cast<double>(p.x) * q.x + static_cast<double>(p.y) * q.y) +
                 (static_cast<double>(p.z) * q.z + static_cast<double>(p.w) * q.w);
        }
    } else {
        for (int64_t e = tid; e < a.dkv; e += NTH) x += static_cast<double>(s[e]) * d[e];
    }
    auto total = [&](double v) {  // over the workgroup, the same on every lane
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
        __syncthreads();  // red's previous readers
        if (lane == 0) red[tid >> 6] = v;
        __syncthreads();
        v = 0.0;
#pragma unroll
        for (int w = 0; w < NW; ++w) v += red[w];
        return v;
    };
    x = total(x);
    // the reverse state has yet to pass the decay behind the segment
    if (!last) x *= exp(static_cast<double>(max(a.la[a.la_tok ? hi * a.H + h : h], LA_MIN)));
    double sum = 0.0;
    const float *uq = a.uq + static_cast<int64_t>(h) * a.tokens, *uk = a.uk + static_cast<int64_t>(h) * a.tokens;
    const float *um = a.m + static_cast<int64_t>(h) * a.tokens;
    for (int64_t top = lo + (hi - lo + 63) / 64 * 64; top > lo; top -= NTH) {
        const int64_t t = top - 1 - tid;
        const bool live = t >= lo && t < hi;
        const double upto = wave_prefix(live ? static_cast<double>(uq[t]) - static_cast<double>(uk[t]) : 0.0);
        double pairs = wave_prefix(live ? static_cast<double>(um[t]) : 0.0);
        if (a.half) {
            const double first = __shfl(pairs, 31);
            if (lane >= 32) pairs -= first;
        }
        __syncthreads();  // red's previous readers
        if (lane == 63) red[tid >> 6] = upto;
        __syncthreads();
        double before = 0.0, all = 0.0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            before += w < (tid >> 6) ? red[w] : 0.0;
            all += red[w];
        }
        if (live) {
            const double g = x + before + upto + pairs;
            if (a.la_tok) a.d_la[t * a.H + h] = static_cast<float>(g);
            sum += g;
        }
        x += all;
    }
    if (!a.la_tok) {
        sum = total(sum);
        if (tid == 0) a.part[sh] = sum;
    }
}

// Per-head decays: the segments' sums, always in the same order.
__global__ void __launch_bounds__(64) decay_sum_kernel(const double *part, const int *nsegs, int64_t segs, int H,
                                                      float *d_la) {
    const int h = blockIdx.x, lane = threadIdx.x;
    const int64_t n = nsegs ? *nsegs : segs;
    double s = 0.0;
    for (int64_t i = lane; i < n; i += 64) s += part[i * H + h];
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o);
    if (lane == 0) d_la[h] = static_cast<float>(s);
}

// The plan of up to 1024 packed sequences in one launch (the two of
// varlen.hip else): every workgroup counts the segments of all sequences and
// fills its share of the segment table.
__global__ void __launch_bounds__(1024) plan_kernel(const int32_t *cu, int n, int64_t T, int L, int cap, int2 *seq, int *pfx,
                                                   int2 *tab) {
    __shared__ int64_t part[16];
    __shared__ int first[1025], from[1024], to[1024];
    const int i = threadIdx.x, lane = i & 63, wave = i >> 6;
    int64_t lo = 0, hi = 0, sum = 0;
    if (i < n) {
        lo = min(max(static_cast<int64_t>(cu[i]), int64_t(0)), T);
        hi = min(max(static_cast<int64_t>(cu[i + 1]), lo), T);
        sum = (hi - lo + L - 1) / L;
        from[i] = static_cast<int>(lo);
        to[i] = static_cast<int>(hi);
    }
    const int64_t mine = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t x = __shfl_up(sum, o);
        if (lane >= o) sum += x;
    }
    if (lane == 63) part[wave] = sum;
    __syncthreads();
    for (int w = 0; w < wave; ++w) sum += part[w];
    if (i < n) {
        first[i] = static_cast<int>(min(sum - mine, static_cast<int64_t>(cap)));
        if (i == n - 1) first[n] = static_cast<int>(min(sum, static_cast<int64_t>(cap)));
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        if (i < n) {
            seq[i] = make_int2(from[i], to[i]);
            pfx[i] = first[i];
        }
        if (i == 0) pfx[n] = first[n];
    }
    const int total = first[n];
    for (int s = blockIdx.x * 1024 + i; s < total; s += gridDim.x * 1024) {
        int l = 0, r = n - 1;  // the last sequence that starts at or before segment s
        while (l < r) {
            const int mid = (l + r + 1) >> 1;
            if (first[mid] <= s) l = mid;
            else r = mid - 1;
        }
        tab[s] = make_int2(from[l] + L * (s - first[l]), to[l]);
    }
}

// ---- host side

int64_t align256(int64_t x) { return (x + 255) & ~int64_t(255); }

hipError_t launch_plan(const LinArgs &a, int L, char *buf, VarPlan *plan, hipStream_t s) {
    if (a.N > 1024) return launch_varlen_plan(a.cu, a.N, a.T, L, buf, plan, s);
    const int n = static_cast<int>(a.N);
    int2 *seq = reinterpret_cast<int2 *>(buf);
    int *pfx = reinterpret_cast<int *>(buf + align256(a.N * 8));
    int2 *tab = reinterpret_cast<int2 *>(buf + align256(a.N * 8) + align256((a.N + 1) * 4));
    const int64_t cap = varlen_chunk_bound(a.N, a.T, L), blocks = (cap + 1023) / 1024;
    hipLaunchKernelGGL(plan_kernel, dim3(static_cast<unsigned>(blocks < 256 ? blocks : 256)), dim3(1024), 0, s, a.cu, n, a.T, L,
                       static_cast<int>(cap), seq, pfx, tab);
    *plan = VarPlan{seq, pfx, tab};
    return hipGetLastError();
}

struct Cut {
    int L;         // tokens of a segment
    int64_t nseg;  // segments of a batched sequence
    int64_t segs;  // segments in all (packed: the most there can be)
};

Cut cut_of(const LinArgs &a, int64_t L) {
    Cut c;
    c.L = static_cast<int>(L);
    c.nseg = (a.T + L - 1) / L;
    c.segs = a.cu ? varlen_chunk_bound(a.N, a.T, c.L) : a.N * c.nseg;
    return c;
}

// Tokens of a segment, in whole chunks, so that all heads together have at
// most `most` of them (packed sequences: and one more each).
int64_t segment_tokens(const LinArgs &a, int64_t most) {
    const int64_t heads = a.H * (a.cu || a.N < 1 ? 1 : a.N), n = heads < most ? most / heads : 1, C = a.bf16 ? 64 : 32;
    return ((a.T + n - 1) / n + C - 1) / C * C;
}

// Forward: segments where whole chains leave the chip empty, two for each CU.
// Measured (H=16, d=128, bf16), whole chains and segments: 64 chains of 4096
// tokens 194 and 130 us, 112 chains 197 and 206, 128 chains 206 and 230, 192
// chains 274 and 356; 16 chains of 512 tokens 29 and 27 us, of 1024 53 and 30
// (fp32, 256 tokens: 39 and 41; 512: 73 and 43).
Cut fwd_cut(const LinArgs &a) {
    const int64_t heads = a.H * (a.cu ? 1 : a.N);
    if (a.T <= (a.bf16 ? 512 : 256) || heads >= 112) return Cut{0, 1, a.N};
    int64_t L = segment_tokens(a, 512);
    if (L < 96) L = a.bf16 ? 128 : 96;
    if (!a.cu && L >= a.T) return Cut{0, 1, a.N};
    return cut_of(a, L);
}

// Backward: always through the segments' states, at most 1024 tokens apart,
// which bounds how far the differences of the decay's gradient are summed.
// One gradient sweep of eight waves fills a CU (64 chains of 4096 tokens, the
// whole call: 372 us, with segments of 2048 or 512 tokens 406 and 412), or two
// of four waves.
Cut bwd_cut(const LinArgs &a) {
    const int64_t L = segment_tokens(a, a.dk > 64 || a.dv > 64 ? 256 : 512);
    return cut_of(a, L < 64 ? 64 : L > 1024 ? 1024 : L);
}

template <class T, int DX, int NCW, int NT, int KSP, int MODE, int NP, int NS, int NU>
hipError_t launch_shape(SweepArgs a, bool vec, hipStream_t s) {
    using Sh = Shape<T, DX, NCW, NT, KSP>;
    a.ncb = (a.dz + Sh::WC - 1) / Sh::WC;
    const int64_t blocks = xcd_blocks(a.segs * a.H, a.ncb);
    if (blocks <= 0) return hipSuccess;
    if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
    constexpr size_t lds = Sh::bytes(MODE, NP);
    auto go = [&](auto kernel) {
        static_assert(lds <= 160 * 1024, "LDS of a CU");
        if (lds > 64 * 1024) {
            const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
            if (e != hipSuccess) return e;
        }
        hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(blocks)), dim3(64 * Sh::NW), lds, s, a);
        return hipGetLastError();
    };
    if (vec) return go(sweep_kernel<T, DX, NCW, NT, KSP, MODE, NP, NS, NU, true>);
    return go(sweep_kernel<T, DX, NCW, NT, KSP, MODE, NP, NS, NU, false>);
}

// The sweep's shapes: columns of a workgroup and how its waves share them.
//   WIDE   128 columns, four waves of 32, two workgroups a CU
//   TALL   128 columns, eight waves of 16: fewer registers a wave, for the
//          sweeps that hold more operands
//   SPLIT  64 columns, four pairs of waves, each pair sharing 16 columns and
//          taking half of the channels: eight waves on half of a head, where
//          whole heads would leave CUs empty
// and up to 64 columns four waves of 16.  Whole chains, SPLIT, TALL and WIDE:
//   bf16, 4096 tokens, 128 x 128   128 chains 204 271 468 us, 144 385 272 472,
//                                  256 407 312 503, 512 815 615 720
//   bf16, 4096 tokens,  64 x 128   128 chains 163 204 204, 256 275 235 218,
//                                  512 545 465 383
//   fp32, 1024 tokens, 128 x 128   128 chains 145 209 212, 256 254 219 216,
//                                  512 500 431 377
// In bf16 above 64 channels WIDE's update in three parts takes more than its
// 256 registers (35 spilled, and their loads wait behind the next chunk's
// rows), so TALL stands in for it.  Segments (an update in two parts, 8
// spilled), WIDE and TALL: 65536 tokens on 16 heads 402 and 430 us, fp32 7777
// packed tokens on 5 heads 79 and 87.  The gradients (WIDE would not fit their
// registers) are TALL.
enum Form { WIDE, TALL, SPLIT };

template <class T, int DX, int MODE, int NP, int NS, int NU>
hipError_t launch_width(const SweepArgs &a, Form form, bool vec, hipStream_t s) {
    if (a.dz <= 64) return launch_shape<T, DX, 4, 1, 1, MODE, NP, NS, NU>(a, vec, s);
    if constexpr (MODE == OUT) {
        if (form == SPLIT) return launch_shape<T, DX, 4, 1, 2, MODE, NP, NS, NU>(a, vec, s);
        if constexpr (sizeof(T) == 4 || DX == 64 || NU < 3)
            if (form == WIDE) return launch_shape<T, DX, 4, 2, 1, MODE, NP, NS, NU>(a, vec, s);
    }
    return launch_shape<T, DX, 8, 1, 1, MODE, NP, NS, NU>(a, vec, s);
}

template <class T, int MODE, int NP, int NS, int NU>
hipError_t launch_sweep(const SweepArgs &a, Form form, bool vec, hipStream_t s) {
    if (a.dx > 64) return launch_width<T, 128, MODE, NP, NS, NU>(a, form, vec, s);
    return launch_width<T, 64, MODE, NP, NS, NU>(a, form, vec, s);
}

template <int MODE, int NP, int NS, int NU>
hipError_t launch_typed(const LinArgs &l, const SweepArgs &a, Form form, bool vec, hipStream_t s) {
    if (l.bf16) return launch_sweep<__bf16, MODE, NP, NS, NU>(a, form, vec, s);
    return launch_sweep<float, MODE, 1, 1, 1>(a, form, vec, s);
}

SweepArgs sweep_of(const LinArgs &l, const Cut &c, const VarPlan *vp) {
    SweepArgs a = {};
    a.la = l.la;
    a.T = l.T;
    a.tokens = l.cu ? l.T : l.N * l.T;
    a.H = static_cast<int>(l.H);
    a.la_tok = l.la_tok;
    a.nseg = static_cast<int>(c.nseg);
    a.L = c.L ? c.L : static_cast<int>(l.T < 1 ? 1 : l.T);
    a.segs = c.segs;
    a.cu = l.cu;
    if (vp) {
        a.tab = vp->tab;
        a.nsegs = vp->pfx + l.N;
    }
    a.p_scale = a.u_scale = a.s_scale = 1.f;
    return a;
}

// Bytes of one access to rows of d elements at these addresses.
int granularity(const LinArgs &l, int64_t d, std::initializer_list<const void *> ps) {
    const int esz = l.bf16 ? 2 : 4;
    int g = d * esz % 16 == 0 ? 16 : d * esz % 4 == 0 ? 4 : 2;
    for (const void *p : ps) {
        const uintptr_t u = reinterpret_cast<uintptr_t>(p);
        if (g == 16 && u % 16 != 0) g = 4;
        if (g == 4 && u % 4 != 0) g = 2;
    }
    return g;
}

hipError_t launch_scans(const Scans &a, int n, hipStream_t s) {
    const int v = a.s[0].dkv % 4 == 0 ? 4 : 1;
    const int64_t states = a.s[0].N * a.s[0].H;
    if (states <= 0) return hipSuccess;
    if (states > 0x7fffffffLL) return hipErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(states), static_cast<unsigned>((a.s[0].dkv + 256 * v - 1) / (256 * v)), n);
    if (v == 4)
        hipLaunchKernelGGL(segment_scan_kernel<4>, grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL(segment_scan_kernel<1>, grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

template <class K>
hipError_t launch_lds(K kernel, int64_t blocks, int threads, size_t lds, const Sweeps &a, hipStream_t s) {
    if (blocks <= 0) return hipSuccess;
    if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(blocks)), dim3(threads), lds, s, a);
    return hipGetLastError();
}

// Both of the backward's launches for head sizes that share one shape: up to
// 64 channels, or more, on both sides.
template <class T, int D, bool VEC>
hipError_t launch_states(const Sweeps &a, hipStream_t s) {
    constexpr int NCW = D / 16;
    using Sh = Shape<T, D, NCW, 1, 1>;
    const int64_t groups = (a.s[0].segs * a.s[0].H + 7) / 8 * 8;
    return launch_lds(state_pair_kernel<T, D, NCW, VEC>, 2 * groups, 64 * NCW, Sh::bytes(STATE, 1), a, s);
}
template <class T, int D, bool VEC>
hipError_t launch_gradients(const Sweeps &a, hipStream_t s) {
    constexpr int NCW = D / 16;
    using Sh = Shape<T, D, NCW, 1, 1>;
    const int64_t groups = (a.s[0].segs * a.s[0].H + SWEEP_GROUP - 1) / SWEEP_GROUP * SWEEP_GROUP;
    return launch_lds(gradient_kernel<T, D, NCW, VEC>, 3 * groups, 64 * NCW, Sh::bytes(OUTM, sizeof(T) == 2 ? 2 : 1), a, s);
}
template <class T, int D>
hipError_t launch_joint(bool states, const Sweeps &a, bool vec, hipStream_t s) {
    if (states) return vec ? launch_states<T, D, true>(a, s) : launch_states<T, D, false>(a, s);
    return vec ? launch_gradients<T, D, true>(a, s) : launch_gradients<T, D, false>(a, s);
}
hipError_t launch_joint(const LinArgs &l, bool states, const Sweeps &a, bool vec, hipStream_t s) {
    if (l.dk > 64) return l.bf16 ? launch_joint<__bf16, 128>(states, a, vec, s) : launch_joint<float, 128>(states, a, vec, s);
    return l.bf16 ? launch_joint<__bf16, 64>(states, a, vec, s) : launch_joint<float, 64>(states, a, vec, s);
}

struct Bump {
    char *p;
    int64_t used = 0;
    template <class X>
    X *take(int64_t n) {
        X *r = p ? reinterpret_cast<X *>(p + used) : nullptr;
        used += align256(n * static_cast<int64_t>(sizeof(X)));
        return r;
    }
};

struct FwdSpace {
    float *tab;
    double *tot;
    char *plan;
    int64_t bytes;
};

FwdSpace fwd_space(const LinArgs &a, const Cut &c, void *ws) {
    Bump b{static_cast<char *>(ws)};
    FwdSpace f = {};
    if (c.L) {
        f.tab = b.take<float>(c.segs * a.H * a.dk * a.dv);
        f.tot = b.take<double>(c.segs * a.H);
        if (a.cu) f.plan = b.take<char>(static_cast<int64_t>(varlen_plan_bytes(a.N, a.T, c.L)));
    }
    f.bytes = b.used;
    return f;
}

struct BwdSpace {
    float *s_tab, *d_tab, *s_fin, *uq, *uk, *um;
    double *s_tot, *d_tot, *part;
    char *plan;
    int64_t bytes;
};

BwdSpace bwd_space(const LinArgs &a, const Cut &c, void *ws) {
    Bump b{static_cast<char *>(ws)};
    BwdSpace f = {};
    const int64_t dkv = a.dk * a.dv, tokens = a.cu ? a.T : a.N * a.T;
    f.s_tab = b.take<float>(c.segs * a.H * dkv);
    f.d_tab = b.take<float>(c.segs * a.H * dkv);
    f.s_fin = b.take<float>(a.N * a.H * dkv);
    f.s_tot = b.take<double>(c.segs * a.H);
    f.d_tot = b.take<double>(c.segs * a.H);
    f.part = b.take<double>(c.segs * a.H);
    f.uq = b.take<float>(a.H * tokens);
    f.uk = b.take<float>(a.H * tokens);
    f.um = b.take<float>(a.H * tokens);
    if (a.cu) f.plan = b.take<char>(static_cast<int64_t>(varlen_plan_bytes(a.N, a.T, c.L)));
    f.bytes = b.used;
    return f;
}

}  // namespace

bool linear_fits(const LinArgs &a, bool backward) {
    const Cut c = backward ? bwd_cut(a) : fwd_cut(a);
    // workgroups of up to 1024 lanes a segment and head, three of 512 in the
    // gradient sweeps; 256 a state along the scan's first axis
    const int64_t most = INT64_C(1) << 32, sh = c.segs * a.H + SWEEP_GROUP;
    return sh < most / (backward ? 1536 : 1024) && a.N * a.H < most / 4096;
}

size_t linear_fwd_workspace(const LinArgs &a) { return static_cast<size_t>(fwd_space(a, fwd_cut(a), nullptr).bytes); }
size_t linear_bwd_workspace(const LinArgs &a) { return static_cast<size_t>(bwd_space(a, bwd_cut(a), nullptr).bytes); }

hipError_t launch_linear_fwd(const LinArgs &l, void *ws, hipStream_t s) {
    const Cut c = ws ? fwd_cut(l) : Cut{0, 1, l.N};
    hipError_t e;
    VarPlan vp;
    const FwdSpace f = fwd_space(l, c, ws);
    const bool cut = c.L > 0;
    if (cut && l.cu && (e = launch_plan(l, c.L, f.plan, &vp, s)) != hipSuccess) return e;
    SweepArgs a = sweep_of(l, c, cut && l.cu ? &vp : nullptr);
    a.x = l.q;
    a.y = l.k;
    a.z = l.v;
    a.dx = static_cast<int>(l.dk);
    a.dz = static_cast<int>(l.dv);
    a.out = l.o;
    a.s_in = l.s0;
    a.s_out = l.s_out;
    a.gx = granularity(l, l.dk, {l.q, l.k});
    a.gz = granularity(l, l.dv, {l.v, l.o});
    const bool vec = a.gx == 16 && a.gz == 16;
    if (cut) {
        SweepArgs st = a;
        st.s_in = nullptr;
        st.s_out = f.tab;
        st.tot = f.tot;
        if ((e = launch_typed<STATE, 1, 1, 3>(l, st, TALL, vec, s)) != hipSuccess) return e;
        const ScanArgs sc = {f.tab, f.tot, l.s0, l.s_out, l.cu ? vp.pfx : nullptr, l.cu ? vp.seq : nullptr, l.la, l.N, l.T,
                       l.dk * l.dv, a.H, a.nseg, 0, l.la_tok};
        if ((e = launch_scans({{sc, {}}}, 1, s)) != hipSuccess) return e;
        a.s_in = f.tab;
        a.s_out = nullptr;
    }
    a.p_scale = a.s_scale = l.scale;
    // whole chains also give the final state: their updates keep 24 bits
    if (cut) return launch_typed<OUT, 2, 2, 2>(l, a, WIDE, vec, s);
    return launch_typed<OUT, 2, 2, 3>(l, a, l.N * l.H > 128 ? WIDE : SPLIT, vec, s);
}

hipError_t launch_linear_bwd(const LinArgs &l, void *ws, hipStream_t s) {
    const Cut c = bwd_cut(l);
    const BwdSpace f = bwd_space(l, c, ws);
    hipError_t e;
    VarPlan vp;
    if (l.cu && (e = launch_plan(l, c.L, f.plan, &vp, s)) != hipSuccess) return e;
    SweepArgs base = sweep_of(l, c, l.cu ? &vp : nullptr);
    base.ncb = 1;
    const int dk = static_cast<int>(l.dk), dv = static_cast<int>(l.dv);
    const int gk = granularity(l, dk, {l.q, l.k, l.dq, l.dk_out}), gv = granularity(l, dv, {l.v, l.d_o, l.dv_out});
    const bool vec = gk == 16 && gv == 16, joint = (dk > 64) == (dv > 64);

    // what the segments add to the state, and in reverse to its gradient
    Sweeps w = {{base, base, base}};
    w.s[0].y = l.k; w.s[0].z = l.v; w.s[0].dx = dk; w.s[0].dz = dv; w.s[0].gx = gk; w.s[0].gz = gv;
    w.s[0].s_out = f.s_tab; w.s[0].tot = f.s_tot;
    w.s[1] = w.s[0];
    w.s[1].y = l.q; w.s[1].z = l.d_o; w.s[1].rev = 1; w.s[1].u_scale = l.scale;
    w.s[1].s_out = f.d_tab; w.s[1].tot = f.d_tot;
    if (joint) {
        if ((e = launch_joint(l, true, w, vec, s)) != hipSuccess) return e;
    } else {
        for (int i = 0; i < 2; ++i)
            if ((e = launch_typed<STATE, 1, 1, 3>(l, w.s[i], TALL, vec, s)) != hipSuccess) return e;
    }
    Scans sc;
    sc.s[0] = {f.s_tab, f.s_tot, l.s0, f.s_fin, l.cu ? vp.pfx : nullptr, l.cu ? vp.seq : nullptr, l.la, l.N, l.T,
               l.dk * l.dv, base.H, base.nseg, 0, l.la_tok};
    sc.s[1] = sc.s[0];
    sc.s[1].tab = f.d_tab; sc.s[1].tot = f.d_tot; sc.s[1].init = l.d_sT; sc.s[1].fin = l.d_s0; sc.s[1].rev = 1;
    if ((e = launch_scans(sc, 2, s)) != hipSuccess) return e;

    w = {{base, base, base}};
    SweepArgs &q = w.s[0], &k = w.s[1], &v = w.s[2];
    q.x = l.d_o; q.y = l.v; q.z = l.k; q.dx = dv; q.dz = dk; q.gx = gv; q.gz = gk;
    q.s_t = 1;
    k = q;
    q.out = l.dq; q.w = l.q; q.u = f.uq; q.m = f.um;
    q.s_in = f.s_tab;
    q.p_scale = q.s_scale = l.scale;
    k.x = l.v; k.y = l.d_o; k.z = l.q;
    k.out = l.dk_out; k.w = l.k; k.u = f.uk;
    k.s_in = f.d_tab; k.rev = 1;
    k.p_scale = k.u_scale = l.scale;
    v.x = l.k; v.y = l.q; v.z = l.d_o; v.dx = dk; v.dz = dv; v.gx = gk; v.gz = gv;
    v.out = l.dv_out;
    v.s_in = f.d_tab; v.rev = 1;
    v.p_scale = v.u_scale = l.scale;
    if (joint) {
        if ((e = launch_joint(l, false, w, vec, s)) != hipSuccess) return e;
    } else {
        if ((e = launch_typed<OUTM, 2, 3, 3>(l, q, TALL, vec, s)) != hipSuccess) return e;
        if ((e = launch_typed<OUTU, 2, 3, 3>(l, k, TALL, vec, s)) != hipSuccess) return e;
        if ((e = launch_typed<OUT, 2, 2, 2>(l, v, TALL, vec, s)) != hipSuccess) return e;
    }

    DecayArgs d = {f.uq, f.uk, f.um, f.s_tab, f.d_tab, f.s_fin, l.la, l.d_la, f.part, l.cu ? vp.tab : nullptr,
                   l.cu ? vp.seq : nullptr, l.cu ? vp.pfx : nullptr, l.N, l.T, base.tokens, c.segs, l.dk * l.dv, base.H,
                   base.nseg, c.L, l.la_tok, !l.bf16};
    if (c.segs * l.H > 0) {
        // lanes for the segment's tokens: 576 segments of at most 512 tokens 16 us with 1024 lanes
        // (the chip holds 512 such workgroups) and 8 with 256, 256 of 1024 tokens 14 and 20
        if (c.L <= 512)
            hipLaunchKernelGGL(decay_grad_kernel<256>, dim3(static_cast<unsigned>(c.segs * l.H)), dim3(256), 0, s, d);
        else
            hipLaunchKernelGGL(decay_grad_kernel<1024>, dim3(static_cast<unsigned>(c.segs * l.H)), dim3(1024), 0, s, d);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (!l.la_tok) {
        hipLaunchKernelGGL(decay_sum_kernel, dim3(static_cast<unsigned>(l.H)), dim3(64), 0, s, f.part,
                           l.cu ? vp.pfx + l.N : nullptr, c.segs, base.H, l.d_la);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace gdn2
