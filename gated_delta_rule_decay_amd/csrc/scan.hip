// scan.hip -- a gated linear recurrence over channels, forward and backward.
//
// Here: what is prepared before a launch, and the decode step.  The forward is
// in scan_fwd.hip, the backward in scan_bwd.hip, what they share in scan_tile.h.
#include "scan_tile.h"

namespace gdn2 {
namespace scan {
namespace {

// The shared words, the sequence index of each token, and the states of empty
// sequences, which pass through: 5 us before the scan's own launch, in which no
// workgroup knows that all others have seen cleared words.
__global__ void __launch_bounds__(256) scan_plan_kernel(Chain ch, int64_t words, const int32_t *cu, int n, int T, int D,
                                                       const float *from, float *to) {
    const int64_t step = static_cast<int64_t>(gridDim.x) * 256, first = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (ch.tiles > 1) {
        if (first < COUNTER_WORDS) ch.counters[first] = 0;
        for (int64_t i = first; i < words; i += step) ch.maps[i] = NOT_YET;
    }
    if (!cu) return;
    for (int64_t i = first; i < static_cast<int64_t>(T) + 2; i += step) {
        const int t = static_cast<int>(i - 1);
        if (t < 0 || t >= T) {
            ch.seq[i] = 0;
            continue;
        }
        int lo = 0, hi = n;  // the last sequence that starts at or before t
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= t) lo = mid + 1;
            else hi = mid;
        }
        ch.seq[i] = lo > 0 && t < cu[lo] ? lo : 0;
    }
    if (!to) return;
    for (int64_t i = first; i < static_cast<int64_t>(n) * D; i += step) {
        const int q = static_cast<int>(i / D);
        const int lo = min(max(cu[q], 0), T), hi = min(max(cu[q + 1], lo), T);
        if (hi == lo && to != from) to[i] = from ? from[i] : 0.f;
    }
}

// One token: bound by the launch (256 sequences of 2048 channels: 3.6 us on the
// GPU, 7 from call to call), and by HBM with many (4096: 20 us; not in whole
// vectors 22).
template <class T, class G, int VE>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanStepArgs a) {
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (256 * VE);
    const int n = static_cast<int>(a.n - first < 256 * VE ? a.n - first : 256 * VE);
    const unsigned i = threadIdx.x * VE;
    const auto bs = buffer<float>(a.state, first, n);
    Row<T, VE> x;
    Row<G, VE> g;
    Row<float, VE> s;
    x.load(buffer<T>(a.x, first, n), i * sizeof(T));
    g.load(buffer<G>(a.gate, first, n), i * sizeof(G));
    s.load(bs, i * 4);
    float h[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) {
        const float v = a.logits ? small_of_logit(g[e]) : small_of_log(g[e]);
        const float u = a.comp ? rest_of(v) * x[e] : x[e];
        // of a decay near 1 by its complement: a state passes this rounding once a token
        h[e] = __float_as_int(v) < 0 ? s[e] + (u - rest_of(v) * s[e]) : v * s[e] + u;
    }
    store_row<float, VE>(bs, i * 4, h);
    store_row<T, VE>(buffer<T>(a.y, first, n), i * sizeof(T), h);
}

template <class F>
hipError_t by_type(int bf16, int gate_bf16, F f) {
    using B = uint16_t;
    if (bf16) return gate_bf16 ? f(B(), B()) : f(B(), float());
    return gate_bf16 ? f(float(), B()) : f(float(), float());
}

int64_t chains_of(const ScanArgs &a) { return (a.cu ? 1 : a.N) * ((a.D + CW - 1) / CW); }
int64_t tiles_of(const ScanArgs &a) { return (a.T + ROWS - 1) / ROWS; }
size_t align256(size_t n) { return (n + 255) / 256 * 256; }

size_t seq_bytes(const ScanArgs &a) { return a.cu ? align256((static_cast<size_t>(a.T) + 2) * 4) : 0; }
int64_t words_of(const ScanArgs &a) {
    const int64_t tiles = tiles_of(a);
    return tiles > 1 ? chains_of(a) * (tiles + tiles / RUN + tiles / SPAN) * CW : 0;
}

}  // namespace

hipError_t prepare(const ScanArgs &a, void *ws, const float *from, float *to, Chain &ch, hipStream_t s) {
    char *p = static_cast<char *>(ws);
    ch.tiles = static_cast<int>(tiles_of(a));
    ch.chains = static_cast<int>(chains_of(a));
    ch.share = (ch.chains + GROUPS - 1) / GROUPS;
    ch.groups = (ch.chains + ch.share - 1) / ch.share;
    ch.seq = reinterpret_cast<int *>(p);
    p += seq_bytes(a);
    ch.counters = reinterpret_cast<unsigned *>(p);
    p += align256(COUNTER_WORDS * 4);
    ch.maps = reinterpret_cast<uint64_t *>(p);
    ch.runs = ch.maps + static_cast<int64_t>(ch.chains) * ch.tiles * CW;
    ch.states = ch.runs + static_cast<int64_t>(ch.chains) * (ch.tiles / RUN) * CW;
    const int64_t words = words_of(a);
    if (!a.cu && !words) return hipSuccess;
    int64_t work = a.cu ? a.T + 2 : 0;
    if (a.cu && to && a.N * a.D > work) work = a.N * a.D;
    if (words > work) work = words;
    if (work < COUNTER_WORDS) work = COUNTER_WORDS;
    work = (work + 255) / 256;
    hipLaunchKernelGGL(scan_plan_kernel, dim3(static_cast<unsigned>(work < 2048 ? work : 2048)), dim3(256), 0, s, ch, words, a.cu,
                       static_cast<int>(a.N), static_cast<int>(a.T), static_cast<int>(a.D), from, to);
    return hipGetLastError();
}

}  // namespace scan

using namespace scan;

bool scan_fits(const ScanArgs &a) {
    const int64_t tiles = tiles_of(a) > 0 ? tiles_of(a) : 1, blocks = (a.D + CW - 1) / CW;
    // with one tile each, chains are workgroups (rounded up to whole groups) of up
    // to 1024 lanes, and a launch of 2^32 lanes is cut short without an error
    const int64_t most = (INT64_C(1) << 22) - GROUPS;
    return blocks <= most / (a.cu || a.N == 0 ? 1 : a.N) && chains_of(a) < most &&
           chains_of(a) <= INT32_MAX / tiles && a.D < (INT64_C(1) << 21) &&  // 31-bit offsets within a tile
           (!a.cu || a.N * a.D < (INT64_C(1) << 29));                        // and within packed states
}

size_t scan_workspace(const ScanArgs &a) {
    const int64_t words = words_of(a);
    return seq_bytes(a) + (words ? align256(COUNTER_WORDS * 4) + static_cast<size_t>(words) * 8 : 0);
}

hipError_t launch_scan_step(const ScanStepArgs &a, hipStream_t s) {
    const bool vec = a.n % 8 == 0 && aligned(a.x) && aligned(a.gate) && aligned(a.y) && aligned(a.state);
    return by_type(a.bf16, a.gate_bf16, [&](auto t, auto g) {
        using T = decltype(t);
        using G = decltype(g);
        const int64_t lanes = vec ? a.n / 8 : a.n, grid = (lanes + 255) / 256;  // scan_fits: under 2^28 lanes
        if (vec) hipLaunchKernelGGL((scan_step_kernel<T, G, 8>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, a);
        else hipLaunchKernelGGL((scan_step_kernel<T, G, 1>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, a);
        return hipGetLastError();
    });
}

}  // namespace gdn2
