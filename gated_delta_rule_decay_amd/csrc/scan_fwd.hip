// scan_fwd.hip -- the gated scan over whole sequences, see scan_tile.h.
#include "scan_tile.h"

namespace gdn2 {
namespace scan {
namespace {

// Lanes of a workgroup.  Of single elements 512 lanes fit a CU twice (8 x 4096
// tokens of 2047 bf16 channels: 151 us, with 1024 lanes 184; 4 x 4096 of 1023 in
// fp32 54 and 59); packed, with what each token is, they would spill.
template <int VE, bool PACKED>
constexpr int lanes_of() { return VE > 1 ? 256 : PACKED ? 1024 : 512; }

// Workgroups of a CU.  Three, whose registers hold the next tile as well; packed
// tiles of 8 bytes an element would spill 9 of them (7 sequences, 32768 tokens of
// 2048 channels: fp32 206 us with two, 209 with three; bf16 with fp32 gates 172
// and 157, bf16 alone 149 and 137).
template <class T, class G, bool PACKED>
constexpr int per_cu() { return PACKED && sizeof(T) + sizeof(G) > 6 ? 2 : 3; }

template <class T, class G, int VE, int FORM, bool PACKED>
__global__ void __launch_bounds__((lanes_of<VE, PACKED>()), (VE > 1 ? per_cu<T, G, PACKED>() : 4)) scan_fwd_kernel(ScanArgs a, Chain ch) {
    using Q = Lanes<VE, lanes_of<VE, PACKED>()>;
    constexpr int K = Q::K, PARTS = Q::PARTS;
    __shared__ float2 s_map[Q::GRP][Q::ROW];  // groups' maps, then .y the state that enters
    __shared__ float s_rest[Q::GRP][Q::ROW];
    __shared__ float2 s_part[PARTS][CW], s_maps[PARTS][CW], s_runs[PARTS][CW];
    __shared__ float s_start[CW];
    __shared__ unsigned s_take[2];
    const int blocks = static_cast<int>((a.D + CW - 1) / CW), states = PACKED ? static_cast<int>(a.N) : 1;
    const int l = threadIdx.x % Q::LPR, g = threadIdx.x / Q::LPR;
    const int jc = threadIdx.x % CW, jp = __builtin_amdgcn_readfirstlane(threadIdx.x / CW);  // place and part in the joint
    const unsigned D = static_cast<unsigned>(a.D);
    const Form<FORM> form(a);

    // of a tile, as loaded
    Row<T, VE> x[K];
    Row<G, VE> gt[K];
    Rows<K, PACKED> ahead;
    auto fetch = [&](const Spot &p) {
        const unsigned c = p.cb + l * VE, lane = g * K * D + c;
        const int64_t base = p.row * a.D;
        const auto bx = buffer<T>(a.x, base, p.rows * D), bg = buffer<G>(a.gate, base, p.rows * D);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            x[k].load(bx, (c < D ? lane * sizeof(T) : NOWHERE) + k * D * sizeof(T));
            gt[k].load(bg, (c < D ? lane * sizeof(G) : NOWHERE) + k * D * sizeof(G));
        }
        ahead.load(ch.seq, p.row, g * K, p.rows);
    };

    if (jp == 0) {
        s_take[0] = __builtin_amdgcn_readfirstlane(take(ch, true));
        s_take[1] = __builtin_amdgcn_readfirstlane(take(ch, false));
    }
    __syncthreads();
    int tile = tile_of(ch, __builtin_amdgcn_readfirstlane(s_take[0])), after = tile_of(ch, __builtin_amdgcn_readfirstlane(s_take[1]));
    if (tile < 0) return;
    Spot p = spot_of<PACKED>(ch, a.T, blocks, tile, false);
    fetch(p);
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): in the loop the loads are waited for over the stores behind them
    while (tile >= 0) {
        unsigned next = 0;
        if (jp == 0) next = take(ch, false);
        const unsigned c = p.cb + l * VE, lane = g * K * D + c, c4 = c < D ? 4 * c : NOWHERE;
        const int64_t base = p.row * a.D;
        auto at = [&](int k, unsigned size) { return (c < D ? lane * size : NOWHERE) + k * D * size; };
        float A[K][VE], U[K][VE], F[VE];  // F: the factor of the group's map
        const Rows<K, PACKED> rw = ahead;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            F[e] = 1.f;
            float rest = 0.f;  // its complement, as in Joint
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float v = form.logits ? small_of_logit(gt[k][e]) : small_of_log(gt[k][e]);
                v = rw.live(k) ? v : -0.f;  // a = 1, w = 0
                const float w = rest_of(v), u = form.comp ? w * x[k][e] : x[k][e];
                A[k][e] = decay_of(v);
                U[k][e] = PACKED ? (rw.live(k) ? u : 0.f) : u;  // x behind a sequence's end reads as zero
                rest += w * F[e];
                F[e] *= A[k][e];
                settle(A[k][e]);
                settle(U[k][e]);
            }
            settle(F[e]);
            s_rest[g][Q::place(l, e)] = rest;
        }
        const bool edges = PACKED && rw.edges();
        float h0 = 0.f;
        if (!PACKED && p.step == 0) {  // what the chain starts from
            h0 = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(buffer<float>(a.s0, p.sequence * a.D, a.s0 ? D : 0),
                                                                     4 * (p.cb + Q::channel(anew(jc))), 0, 0));
            settle(h0);  // not waited for elsewhere
        }
        LookBack<Q::LOOK> back;
        back.start(ch, p.chain, p.step, jc, jp);
        const bool marked = a.marks != nullptr && jp == 0;  // the tile's first row is in wave 0
        const auto bm = buffer<float>(a.marks, p.mark * a.D, marked ? D : 0);
        if (PACKED && edges) {  // sequences start: from state0, and from nothing before
            const auto b0 = buffer<float>(a.s0, 0, a.s0 ? states * D : 0);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                Row<float, VE> h0;
                h0.load(b0, rw.state(k, rw.first(k), D, c4));
                float m[VE];
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    m[e] = h0[e];
                    U[k][e] += A[k][e] * m[e];
                }
                // here, not below: another wave may end this sequence, and state_out may be state0
                if (k == 0) store_row<float, VE>(bm, only((g == 0) & rw.first(0), c4), m);
            }
        }
        {
            float cu[VE];
            bool starts = false;  // whether a sequence does within the group
#pragma unroll
            for (int k = 0; k < K; ++k) starts = starts | rw.first(k);
#pragma unroll
            for (int e = 0; e < VE; ++e) cu[e] = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float u = A[k][e] * cu[e] + U[k][e];
                    cu[e] = rw.first(k) ? U[k][e] : u;
                }
#pragma unroll
            for (int e = 0; e < VE; ++e) s_map[g][Q::place(l, e)] = make_float2(PACKED ? with_mark(F[e], starts) : F[e], cu[e]);
        }
        __syncthreads();
        if (jp == 0) s_take[0] = __builtin_amdgcn_readfirstlane(next);
        {
            Joint<PACKED> m;
#pragma unroll
            for (int i = 0; i < Q::PER; ++i) {
                const float2 n = s_map[jp * Q::PER + i][jc];
                m.then(fabsf(n.x), s_rest[jp * Q::PER + i][jc], n.y, PACKED && has_mark(n.x));
            }
            s_part[jp][jc] = m.map();
        }
        __syncthreads();
        tile = after;
        after = tile_of(ch, __builtin_amdgcn_readfirstlane(s_take[0]));
        float h = h0;
        if (ch.tiles > 1) {
            Joint<PACKED> m;
            if (jp == 0)
#pragma unroll
                for (int i = 0; i < PARTS; ++i) m.then(s_part[i][jc]);
            h = enter<PACKED, PARTS, Q::LOOK>(ch, back, p.chain, p.step, jc, jp, m.map(), h0, s_maps, s_runs, s_start);
        }
        // The next tile's loads are in flight from here to the next round; behind
        // the last tile they read zeros.  (From before the wait for the words,
        // where a second look waits for them as well: 311 us for 65536 tokens of
        // 2048 channels, from here 296.)
        Spot q = spot_of<PACKED>(ch, a.T, blocks, tile < 0 ? 0 : tile, false);
        if (tile < 0) q.rows = 0;
        fetch(q);
        for (int i = 0; i < jp; ++i) h = pass<PACKED>(s_part[i][jc], h);
#pragma unroll
        for (int i = 0; i < Q::PER; ++i) {
            float2 &m = s_map[jp * Q::PER + i][jc];
            const float through = fabsf(m.x) * h + m.y, next_h = PACKED && has_mark(m.x) ? m.y : through;
            m.y = h;
            h = next_h;
        }
        if (jp == PARTS - 1) leave_state(ch, p.chain, p.step, jc, h);
        __syncthreads();
        const auto by = buffer<T>(a.y, base, p.rows * D);
        float hv[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) hv[e] = s_map[g][Q::place(l, e)].y;
        if (marked) store_row<float, VE>(bm, only((g == 0) & rw.live(0) & !rw.first(0), c4), hv);
        // the state behind the last token, in the wave that holds it; packed: behind each sequence's last
        const bool ends = a.s_out != nullptr && (PACKED ? edges : p.step == ch.tiles - 1);
        const auto bs = PACKED ? buffer<float>(a.s_out, 0, states * D) : buffer<float>(a.s_out, p.sequence * a.D, D);
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float h = A[k][e] * hv[e] + U[k][e];
                hv[e] = rw.first(k) ? U[k][e] : h;
            }
            store_row<T, VE>(by, only(rw.live(k), at(k, sizeof(T))), hv);
            if (ends) store_row<float, VE>(bs, PACKED ? rw.state(k, rw.last(k), D, c4) : only(g * K + k == p.rows - 1, c4), hv);
        }
        p = q;
    }
}

}  // namespace
}  // namespace scan

using namespace scan;

// workgroups that run at once (65536 tokens of 2048 channels: 296 us, with 512 of
// them 310)
constexpr int AT_ONCE = 768;

hipError_t launch_scan_fwd(const ScanArgs &a, void *ws, hipStream_t s) {
    Chain ch = {};
    const hipError_t e = prepare(a, ws, a.s0, a.s_out, ch, s);
    if (e != hipSuccess) return e;
    const bool vec = a.D % 8 == 0 && aligned(a.x) && aligned(a.gate) && aligned(a.y) && aligned(a.s0) && aligned(a.s_out) && aligned(a.marks);
    return by_kind(a, vec, [&](auto t, auto g, auto ve, auto form) {
        using T = decltype(t);
        using G = decltype(g);
        constexpr int VE = decltype(ve)::value, FORM = decltype(form)::value;
        const dim3 grid(grid_of(ch, AT_ONCE)), block(a.cu ? lanes_of<VE, true>() : lanes_of<VE, false>());
        if (a.cu) hipLaunchKernelGGL((scan_fwd_kernel<T, G, VE, FORM, true>), grid, block, 0, s, a, ch);
        else hipLaunchKernelGGL((scan_fwd_kernel<T, G, VE, FORM, false>), grid, block, 0, s, a, ch);
        return hipGetLastError();
    });
}

}  // namespace gdn2
