// scan_bwd.hip -- gradients of the gated scan, see scan_tile.h.
#include "scan_tile.h"

namespace gdn2 {
namespace scan {
namespace {

// Lanes of a workgroup.  Of single elements 1024, one workgroup a CU: twice 512,
// of 16 tokens a lane, spill, and help only where there are many tiles (8 x 4096
// tokens of 2047 bf16 channels 227 us for 264; 4 x 4096 of 1023 in fp32 80 for 79;
// 20000 of 129 28 for 25).
template <int VE>
constexpr int lanes_of() { return VE > 1 ? 256 : 1024; }

// Workgroups of a CU: three, packed two, where three would spill 34 to 72 registers
// (7 sequences, 32768 tokens of 2048 channels: bf16 230 us with two, 288 with
// three; fp32 339 and 452).
template <int VE, bool PACKED>
constexpr int per_cu() { return VE > 1 ? (PACKED ? 2 : 3) : 4; }  // (of single elements: sixteen waves, one workgroup)

template <class T, class G, int VE, int FORM, bool PACKED>
__global__ void __launch_bounds__(lanes_of<VE>(), (per_cu<VE, PACKED>())) scan_bwd_kernel(ScanArgs a, Chain ch) {
    using Q = Lanes<VE, lanes_of<VE>()>;
    constexpr int K = Q::K, PARTS = Q::PARTS;
    // groups' maps: (factor, addend) and (its complement, addend backward), then .y what enters
    __shared__ float2 s_map[Q::GRP][Q::ROW], s_rev[Q::GRP][Q::ROW];
    __shared__ float2 s_part[PARTS][CW], s_rpart[PARTS][CW], s_maps[PARTS][CW], s_runs[PARTS][CW];
    __shared__ float s_start[CW];
    __shared__ unsigned s_take;
    const int blocks = static_cast<int>((a.D + CW - 1) / CW), states = PACKED ? static_cast<int>(a.N) : 1;
    const int l = threadIdx.x % Q::LPR, g = threadIdx.x / Q::LPR;
    const int jc = threadIdx.x % CW, jp = __builtin_amdgcn_readfirstlane(threadIdx.x / CW);
    const unsigned D = static_cast<unsigned>(a.D);
    const Form<FORM> form(a);
    // packed: the states of the sequences
    const auto b0 = buffer<float>(a.s0, 0, PACKED && a.s0 ? states * D : 0), bd = buffer<float>(a.d_sT, 0, PACKED && a.d_sT ? states * D : 0);

    if (jp == 0) s_take = __builtin_amdgcn_readfirstlane(take(ch, true));
    __syncthreads();
    int tile = tile_of(ch, __builtin_amdgcn_readfirstlane(s_take));
    while (tile >= 0) {
        unsigned next = 0;
        if (jp == 0) next = take(ch, false);
        // steps of a chain go from its last tile to its first
        const Spot p = spot_of<PACKED>(ch, a.T, blocks, tile, true);
        const unsigned c = p.cb + l * VE, lane = g * K * D + c, c4 = c < D ? 4 * c : NOWHERE;
        const int64_t base = p.row * a.D;
        auto at = [&](int k, unsigned size) { return (c < D ? lane * size : NOWHERE) + k * D * size; };
        Row<T, VE> x[K], dy[K];
        float V[K][VE];  // decays, see small_of_log
        Rows<K, PACKED> rw;
        // the state that enters the tile, and the gradient that enters the chain
        float h = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(buffer<float>(a.marks, p.mark * a.D, D), 4 * (p.cb + Q::channel(jc)), 0, 0));
        float r0 = 0.f;
        if (!PACKED && p.step == 0)
            r0 = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(buffer<float>(a.d_sT, p.sequence * a.D, a.d_sT ? D : 0), 4 * (p.cb + Q::channel(jc)), 0, 0));
        {
            Row<G, VE> gt[K];
            const auto bx = buffer<T>(a.x, base, p.rows * D), bg = buffer<G>(a.gate, base, p.rows * D), by = buffer<T>(a.dy, base, p.rows * D);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                x[k].load(bx, at(k, sizeof(T)));
                gt[k].load(bg, at(k, sizeof(G)));
                dy[k].load(by, at(k, sizeof(T)));
            }
            rw.load(ch.seq, p.row, g * K, p.rows);
            auto gates = [&](auto f) {
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        V[k][e] = f(gt[k][e]);
                        settle(V[k][e]);
                    }
            };
            if (form.logits) gates([](float y) { return small_of_logit(y); });
            else gates([](float y) { return small_of_log(y); });
        }
        const bool edges = PACKED && rw.edges();
        {
            // maps of the group: the same decays (as in Joint), addends forward and backward
            struct Both { float a = 1.f, rest = 0.f, fu = 0.f, ru = 0.f; };
            bool starts = false, ends = false;  // whether a sequence does, in the group's tokens so far
            auto token = [&](Both &m, int k, int e, float h0, float d0) {
                const float v = rw.live(k) ? V[k][e] : -0.f;  // a = 1, w = 0
                const float f = decay_of(v), w = rest_of(v);
                float u = form.comp ? w * x[k][e] : x[k][e], y = dy[k][e];
                if (PACKED) {  // else what is behind a sequence's end reads as zero
                    u = rw.live(k) ? u + f * h0 : 0.f;
                    y = rw.live(k) ? y + d0 : 0.f;
                }
                const float h = f * m.fu + u, r = m.a * (f * y) + m.ru;
                m.fu = rw.first(k) ? u : h;
                // from right to left: the tokens so far come after this one's r
                m.ru = ends ? m.ru : r;
                m.rest += w * m.a;
                m.a *= f;
            };
            auto put = [&](const Both &m, int e) {
                s_map[g][Q::place(l, e)] = make_float2(PACKED ? with_mark(m.a, starts) : m.a, m.fu);
                s_rev[g][Q::place(l, e)] = make_float2(PACKED ? with_mark(m.rest, ends) : m.rest, m.ru);
            };
            if constexpr (PACKED) {
                Both m[VE];
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    Row<float, VE> h0 = {}, d0 = {};
                    if (edges) {
                        h0.load(b0, rw.state(k, rw.first(k), D, c4));
                        d0.load(bd, rw.state(k, rw.last(k), D, c4));
                    }
#pragma unroll
                    for (int e = 0; e < VE; ++e) token(m[e], k, e, h0[e], d0[e]);
                    starts = starts | rw.first(k);
                    ends = ends | rw.last(k);
                }
#pragma unroll
                for (int e = 0; e < VE; ++e) put(m[e], e);
            } else {
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    Both m;
#pragma unroll
                    for (int k = 0; k < K; ++k) token(m, k, e, 0.f, 0.f);
                    put(m, e);
                }
            }
        }
        __syncthreads();
        if (jp == 0) s_take = __builtin_amdgcn_readfirstlane(next);
        {
            Joint<PACKED> m, n;
#pragma unroll 4
            for (int i = 0; i < Q::PER; ++i) {
                const float2 f = s_map[jp * Q::PER + i][jc], b = s_rev[jp * Q::PER + i][jc];
                m.then(fabsf(f.x), fabsf(b.x), f.y, PACKED && has_mark(f.x));
                n.behind(fabsf(f.x), fabsf(b.x), b.y, PACKED && has_mark(b.x));
            }
            s_part[jp][jc] = m.map();
            s_rpart[jp][jc] = n.map();
        }
        __syncthreads();
        tile = tile_of(ch, __builtin_amdgcn_readfirstlane(s_take));
        float r = r0;
        if (ch.tiles > 1) {
            Joint<PACKED> n;
            if (jp == 0)
#pragma unroll
                for (int i = 0; i < PARTS; ++i) n.behind(s_rpart[i][jc]);
            LookBack<Q::LOOK> back;
            back.start(ch, p.chain, p.step, jc, jp);
            r = enter<PACKED, PARTS, Q::LOOK>(ch, back, p.chain, p.step, jc, jp, n.map(), r0, s_maps, s_runs, s_start);
        }
        for (int i = 0; i < jp; ++i) h = pass<PACKED>(s_part[i][jc], h);
        for (int i = PARTS - 1; i > jp; --i) r = pass<PACKED>(s_rpart[i][jc], r);
#pragma unroll
        for (int i = 0; i < Q::PER; ++i) {
            float2 &m = s_map[jp * Q::PER + i][jc];
            const float through = fabsf(m.x) * h + m.y, next_h = PACKED && has_mark(m.x) ? m.y : through;
            m.y = h;
            h = next_h;
        }
#pragma unroll
        for (int i = Q::PER - 1; i >= 0; --i) {
            float2 &m = s_rev[jp * Q::PER + i][jc];
            const float through = fabsf(s_map[jp * Q::PER + i][jc].x) * r + m.y, next_r = PACKED && has_mark(m.x) ? m.y : through;
            m.y = r;
            r = next_r;
        }
        if (jp == 0) leave_state(ch, p.chain, p.step, jc, r);
        __syncthreads();
        // decoded again below: a and w of all tokens would not fit beside the states
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < VE; ++e) settle(V[k][e]);
        const auto bdx = buffer<T>(a.dx, base, p.rows * D), bdg = buffer<G>(a.d_gate, base, p.rows * D);
        float H[K][VE], rv[VE];  // H: the states that enter the tokens, then what d log a_t takes of them
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            H[0][e] = s_map[g][Q::place(l, e)].y;
            rv[e] = s_rev[g][Q::place(l, e)].y;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (PACKED && edges) {
                Row<float, VE> i;
                i.load(b0, rw.state(k, rw.first(k), D, c4));
#pragma unroll
                for (int e = 0; e < VE; ++e) H[k][e] = rw.first(k) ? i[e] : H[k][e];
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                if (k + 1 < K) H[k + 1][e] = decay_of(V[k][e]) * H[k][e] + (form.comp ? rest_of(V[k][e]) * x[k][e] : x[k][e]);
                if (form.comp) H[k][e] -= x[k][e];
                settle(H[k][e]);
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < VE; ++e) settle(V[k][e]);
        const bool starts = a.d_s0 != nullptr && (PACKED ? edges : p.step == ch.tiles - 1 && jp == 0);
        const auto bs = PACKED ? buffer<float>(a.d_s0, 0, states * D) : buffer<float>(a.d_s0, p.sequence * a.D, D);
#pragma unroll
        for (int k = K - 1; k >= 0; --k) {
            float gx[VE], gl[VE];
            if (PACKED && edges) {
                Row<float, VE> o;
                o.load(bd, rw.state(k, rw.last(k), D, c4));
#pragma unroll
                for (int e = 0; e < VE; ++e) rv[e] = rw.last(k) ? o[e] : rv[e];
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float w = rest_of(V[k][e]), s = dy[k][e] + rv[e];
                rv[e] = rw.live(k) ? decay_of(V[k][e]) * s : rv[e];
                gx[e] = form.comp ? w * s : s;
                gl[e] = rv[e] * H[k][e];
                if (form.logits) gl[e] *= -w;
            }
            store_row<T, VE>(bdx, only(rw.live(k), at(k, sizeof(T))), gx);
            store_row<G, VE>(bdg, only(rw.live(k), at(k, sizeof(G))), gl);
            if (starts) store_row<float, VE>(bs, PACKED ? rw.state(k, rw.first(k), D, c4) : only(g * K + k == 0, c4), rv);
        }
    }
}

}  // namespace
}  // namespace scan

using namespace scan;

// workgroups that run at once, packed two thirds of them: a workgroup takes its
// first tile when it starts, so those that start late find what is left
constexpr int AT_ONCE = 768;

hipError_t launch_scan_bwd(const ScanArgs &a, void *ws, hipStream_t s) {
    Chain ch = {};
    const hipError_t e = prepare(a, ws, a.d_sT, a.d_s0, ch, s);
    if (e != hipSuccess) return e;
    const bool vec = a.D % 8 == 0 && aligned(a.x) && aligned(a.gate) && aligned(a.dy) && aligned(a.dx) && aligned(a.d_gate) &&
                     aligned(a.marks) && aligned(a.s0) && aligned(a.d_sT) && aligned(a.d_s0);
    return by_kind(a, vec, [&](auto t, auto g, auto ve, auto form) {
        using T = decltype(t);
        using G = decltype(g);
        constexpr int VE = decltype(ve)::value, FORM = decltype(form)::value;
        const dim3 grid(grid_of(ch, AT_ONCE)), block(lanes_of<VE>());
        if (a.cu) hipLaunchKernelGGL((scan_bwd_kernel<T, G, VE, FORM, true>), grid, block, 0, s, a, ch);
        else hipLaunchKernelGGL((scan_bwd_kernel<T, G, VE, FORM, false>), grid, block, 0, s, a, ch);
        return hipGetLastError();
    });
}

}  // namespace gdn2
