// Gated linear recurrence for gfx950: per channel d of a sequence
//
//   h_t = a_t h_{t-1} + c_t v_t,   v_t = sigmoid(i_t) x_t,   y_t = h_t
//
// with the decay a_t in (0, 1] and the input's coefficient c_t made from a
// gate f_t: log a = f, c = 1; or a = sigmoid(f), c = 1 - a; or
// log a = rate[d] sigmoid(f), c = sqrt(1 - a^2). reset[t] leaves out h_{t-1}.
//
// k_gated_fwd reads the inputs once. A group of lanes walks its R tokens from a zero state, keeping h and the
// product of the decays; the groups' ends are put together through LDS into the chunk's (a, h), the
// entering state comes from the chunks before (ssd_gated.h), and every h then is its own plus the product
// of the decays times the state that entered its group. Everything is fp32.
#include "ssd_gated.h"

namespace ssd {

// Fills the words with ones and the ticket with zero.
__global__ __launch_bounds__(256) void k_gated_clear(u32x4 *words, int64_t n16) {
    const int64_t hop = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n16; i += hop)
        words[i] = i < 16 ? u32x4{0, 0, 0, 0} : u32x4{~0u, ~0u, ~0u, ~0u};
}

template <typename T, int DECAY, bool IN, int V>
__global__ __launch_bounds__(kGatedThreads, 4) void k_gated_fwd(GatedArgs a) {
    using S = Shape<T, V>;
    constexpr int R = S::R, LPR = S::LPR, GPW = S::GPW;
    constexpr bool kFine = sizeof(T) == 4;
    __shared__ __attribute__((aligned(16))) float ga[S::G][kCols], gh[S::G][kCols];  // the groups' decays and ends, then (gh) entering states
    __shared__ float wa[kGatedWaves][kCols], wh[kGatedWaves][kCols], carry[kCols];
    const Tile tile = take_tile(a.ticket, a.batch, a.cols);
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int j = lane % LPR, g = w * GPW + lane / LPR;
    const int D = (int)a.D, c0 = tile.col * kCols;
    const bool live = c0 + j * V < D;
    const int d = min(c0 + j * V, D - V);  // this lane's channels
    const int t0 = tile.chunk * SSD_GATED_CHUNK + g * R;
    const int n = live ? min(R, (int)a.T - t0) : 0;  // its tokens
    const int64_t row = tile.b * a.T + t0;

    Packed<T, V> x[R], f[R], in[IN ? R : 1];
    uint32_t keep[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        x[r] = {}; f[r] = {};
        if constexpr (IN) in[r] = {};
        keep[r] = ~0u;
        if (r < n) {
            f[r].load(reinterpret_cast<const T *>(a.f) + (row + r) * a.ldf + d);
            x[r].load(reinterpret_cast<const T *>(a.x) + (row + r) * a.ldx + d);
            if constexpr (IN) in[r].load(reinterpret_cast<const T *>(a.i) + (row + r) * a.ldi + d);
        }
    }
    if (a.reset) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (r < n && a.reset[row + r]) keep[r] = 0u;
    }
    float rate[V];
#pragma unroll
    for (int e = 0; e < V; ++e) rate[e] = DECAY == SSD_DECAY_RATE && live ? a.rate[d + e] : 0.f;

    float h[R][V], p[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const Decay q = decay_of<DECAY, kFine, false>(f[r].get(e), rate[e]);
            float v = x[r].get(e);
            if constexpr (IN) v *= sigmoid_of<kFine>(in[r].get(e));
            const float u = q.c * v;
            // tokens behind the end pass the state on
            const float dec = r < n ? q.a : 1.f, add = r < n ? u : 0.f;
            h[r][e] = r ? __builtin_fmaf(dec, masked(h[r ? r - 1 : 0][e], keep[r]), add) : add;
            p[r][e] = masked(r ? p[r ? r - 1 : 0][e] * dec : dec, keep[r]);
        }
#pragma unroll
    for (int e = 0; e < V; ++e) ga[g][j * V + e] = p[R - 1][e], gh[g][j * V + e] = h[R - 1][e];
    __builtin_amdgcn_wave_barrier();
    // this wavefront's groups, a column to a lane
    float qa[GPW], qh[GPW], pa = 1.f, ph = 0.f;
#pragma unroll
    for (int k = 0; k < GPW; ++k) {
        qa[k] = ga[w * GPW + k][lane];
        qh[k] = gh[w * GPW + k][lane];
        ph = pass(qa[k], qh[k], ph);
        pa *= qa[k];
    }
    wa[w][lane] = pa;
    wh[w][lane] = ph;
    __syncthreads();
    if (w == 0) {
        // the channel of this lane's column
        const int base = c0 + lane / V * V, ch = min(base, D - V) + lane % V;
        const bool there = base < D;
        const int64_t at = tile.b * D + ch;
        float first = 0.f;
        if (a.init && there) first = a.init[at];
        if (a.nchunks > 1) {
            float ca = 1.f, chh = 0.f;
#pragma unroll
            for (int k = 0; k < kGatedWaves; ++k) {
                chh = pass(wa[k][lane], wh[k][lane], chh);
                ca *= wa[k][lane];
            }
            const int64_t stride = (int64_t)a.cols * kCols;
            uint64_t *pieces = a.pieces + tile.b * a.nchunks * stride + c0 + lane;
            uint32_t *ends = a.ends + tile.b * a.nchunks * stride + c0 + lane;
            const int k = tile.chunk;
            publish(pieces + k * stride, ca, chh);
            first = entering(pieces, ends, stride, k, first);
            publish(ends + k * stride, pass(ca, chh, first));
        }
        carry[lane] = first;
        if (a.states && there) a.states[(tile.b * a.nchunks + tile.chunk) * D + ch] = first;
    }
    __syncthreads();
    float s = carry[lane];
    for (int k = 0; k < w; ++k) s = pass(wa[k][lane], wh[k][lane], s);
#pragma unroll
    for (int k = 0; k < GPW; ++k) {
        gh[w * GPW + k][lane] = s;
        s = pass(qa[k], qh[k], s);
    }
    if (w == kGatedWaves - 1 && a.final && tile.chunk == a.nchunks - 1) {
        const int base = c0 + lane / V * V;
        if (base < D) a.final[tile.b * D + min(base, D - V) + lane % V] = s;
    }
    __builtin_amdgcn_wave_barrier();
    uint32_t open = ~0u;
    float from[V];
#pragma unroll
    for (int e = 0; e < V; ++e) from[e] = gh[g][j * V + e];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        open &= keep[r];
        float o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = __builtin_fmaf(p[r][e], masked(from[e], open), h[r][e]);
        if (r < n) Packed<T, V>::store(reinterpret_cast<T *>(a.y) + (row + r) * D + d, o);
    }
}

template <typename T>
__device__ __forceinline__ float at(const void *p, int64_t i) {
    return (float)reinterpret_cast<const T *>(p)[i];
}
constexpr int kThreads = 256;

template <typename T, int DECAY, bool IN>
__global__ __launch_bounds__(kThreads) void k_gated_step(GatedStepArgs a) {
    const int64_t k = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (k >= a.rows * a.D) return;
    const int64_t b = k / a.D, d = k - b * a.D;
    const int64_t from = a.parent ? a.parent[b] : b;
    float h = from >= 0 && from < a.src ? a.state_in[from * a.D + d] : 0.f;
    const Decay g = decay_of<DECAY, true, true>(at<T>(a.f, b * a.ldf + d), DECAY == SSD_DECAY_RATE ? a.rate[d] : 0.f);
    float v = at<T>(a.x, b * a.ldx + d);
    if constexpr (IN) v *= gate_of<true>(at<T>(a.i, b * a.ldi + d)).s;
    h = g.a * h + g.c * v;
    a.state_out[k] = h;
    reinterpret_cast<T *>(a.y)[k] = (T)h;
}

GatedPlan gated_plan(int64_t batch, int64_t T, int64_t D, ssd_dtype) {
    GatedPlan p = {};
    p.cols = (D + kCols - 1) / kCols;
    p.nchunks = (T + SSD_GATED_CHUNK - 1) / SSD_GATED_CHUNK;
    const int64_t most = kMostThreads / kGatedThreads;  // one work-group for each
    p.fits = batch == 0 || T == 0 || (batch <= most / p.cols && batch * p.cols <= most / p.nchunks);
    if (!p.fits) return p;
    p.tiles = batch * p.cols * p.nchunks;
    // the ticket, then a chunk's (a, h) and its end for each column
    p.word_bytes = p.nchunks > 1 && p.tiles ? 256 + p.tiles * kCols * 12 : 0;
    p.rate_bytes = batch * p.nchunks * D * 4;
    return p;
}

ssd_status clear_words(GatedArgs &a, const GatedPlan &p, void *workspace, hipStream_t s) {
    a.cols = (int)p.cols;
    if (p.nchunks == 1) return SSD_OK;
    char *ws = static_cast<char *>(workspace);
    a.ticket = reinterpret_cast<uint32_t *>(ws);
    a.pieces = reinterpret_cast<uint64_t *>(ws + 256);
    a.ends = reinterpret_cast<uint32_t *>(ws + 256 + p.tiles * kCols * 8);
    const int64_t n16 = p.word_bytes / 16, blocks = (n16 + 255) / 256;
    return status_of(launch(k_gated_clear, dim3((unsigned)(blocks < 1024 ? blocks : 1024)), dim3(256), s, (u32x4 *)ws, n16));
}

ssd_status launch_gated_fwd(GatedArgs a, const GatedPlan &p, ssd_dtype dtype, int decay, void *workspace, hipStream_t s) {
    const ssd_status st = clear_words(a, p, workspace, s);
    if (st != SSD_OK) return st;
    return pick_gated(dtype, decay, a.i != nullptr, [&](auto t, auto dec, auto in) {
        using T = decltype(t);
        constexpr int DECAY = decltype(dec)::value, V = 16 / (int)sizeof(T);
        constexpr bool IN = decltype(in)::value;
        auto go = [&](auto k) { return status_of(launch(k, dim3((unsigned)p.tiles), dim3(kGatedThreads), s, a)); };
        return a.D >= V ? go(k_gated_fwd<T, DECAY, IN, V>) : go(k_gated_fwd<T, DECAY, IN, 1>);
    });
}

ssd_status launch_gated_step(const GatedStepArgs &a, ssd_dtype dtype, int decay, hipStream_t s) {
    return pick_gated(dtype, decay, a.i != nullptr, [&](auto t, auto dec, auto in) {
        return status_of(launch(k_gated_step<decltype(t), decltype(dec)::value, decltype(in)::value>,
                                dim3((unsigned)((a.rows * a.D + kThreads - 1) / kThreads)), dim3(kThreads), s, a));
    });
}

}  // namespace ssd
