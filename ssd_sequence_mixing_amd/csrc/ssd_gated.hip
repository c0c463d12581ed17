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

// What bounds it: 3 work-groups share a CU, whose vector unit is busy 56 to 67% of the time; a tile's way is its loads, the walk, two
// exchanges through LDS and one look at the chunks before. 4 x 2048 x 4096 in bf16, rates and input gates (268 MB): 69 us,
// 72 with the words' clearing (3.7 TB/s); 16384 x 4096 with resets (403 MB) 99 us together. With the next tile's loads under the
// exchange, at 2 work-groups a CU, they took 77 and 110 where this took 75 and 102.
template <typename T, int DECAY, bool IN, bool RESET, int V>
__global__ __launch_bounds__(kGatedThreads, sizeof(T) == 2 && V > 1 ? 6 : 2) void k_gated_fwd(GatedArgs) {
    Args a = args();
    using S = Shape<T, V>;
    constexpr int R = S::R, LPR = S::LPR, GPW = S::GPW;
    constexpr bool kFine = sizeof(T) == 4;
    __shared__ __attribute__((aligned(16))) float ga[S::G][kCols], gh[S::G][kCols];  // the groups' decays and ends, then (gh) entering states
    // by turns, since a wavefront that is done with a tile writes the next one's while others still read
    __shared__ float wa2[2][kGatedWaves][kCols], wh2[2][kGatedWaves][kCols], carry2[2][kCols];
    __shared__ uint32_t mine;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int j = lane % LPR, g = w * GPW + lane / LPR;
    const int D = (int)a->D;

    Way way(a, &mine);
    for (uint32_t turn = 0; way.chunk < a->nchunks; ++turn) {
    again(a);
    const Tile tile = way.tile((uint32_t)a->cols);
    auto &wa = wa2[turn & 1], &wh = wh2[turn & 1];
    auto &carry = carry2[turn & 1];
    const int c0 = tile.col * kCols;
    const bool live = c0 + j * V < D;
    const int d = min(c0 + j * V, D - V);  // this lane's channels
    const int t0 = tile.chunk * SSD_GATED_CHUNK + g * R;
    const int n = live ? min(R, (int)a->T - t0) : 0;  // its tokens
    const int64_t row0 = tile.b * a->T + (int64_t)tile.chunk * SSD_GATED_CHUNK;
    Packed<T, V> x[R], f[R], in[IN ? R : 1];
    uint8_t marks[RESET ? R : 1];
    {
        const Tokens<T> px(a->x, row0, a->ldx, g * R, d), pf(a->f, row0, a->ldf, g * R, d), pi(a->i, row0, a->ldi, g * R, d);
        const Tokens<uint8_t> pz(a->reset, row0, 1, g * R, 0);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            x[r] = {}; f[r] = {};
            if constexpr (IN) in[r] = {};
            if constexpr (RESET) marks[r] = 0;
            if (r < n) {
                f[r].load(pf[r]);
                x[r].load(px[r]);
                if constexpr (IN) in[r].load(pi[r]);
                if constexpr (RESET) marks[r] = *pz[r];
            }
        }
    }
    float rate[V];
#pragma unroll
    for (int e = 0; e < V; ++e) rate[e] = DECAY == SSD_DECAY_RATE ? base2(a->rate[d + e]) : 0.f;
    uint32_t resets = 0;  // one register for all R
    if constexpr (RESET) {
#pragma unroll
        for (int r = 0; r < R; ++r) resets |= marks[r] ? 1u << r : 0u;
    }
    auto keep = [&](int r) { return resets >> r & 1 ? 0u : ~0u; };
    const uint32_t next = way.ask(a);

    float h[R][V], p[R][V];
    uint32_t open = ~0u;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        open &= keep(r);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            // (behind the last token these are of no use, and of no harm: nobody takes what follows it)
            const Decay q = passed<DECAY, RESET>(decay_of<DECAY, kFine>(f[r].get(e), rate[e]), keep(r));
            float v = x[r].get(e);
            if constexpr (IN) v *= sigmoid_of<kFine>(in[r].get(e));
            const float u = q.c * v;
            h[r][e] = r ? __builtin_fmaf(q.a, cut<RESET>(h[r ? r - 1 : 0][e], keep(r)), u) : u;
            p[r][e] = mark<RESET>(r ? p[r ? r - 1 : 0][e] * q.a : q.a, open);
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) ga[g][j * V + e] = p[R - 1][e], gh[g][j * V + e] = h[R - 1][e];
    __builtin_amdgcn_wave_barrier();
    // this wavefront's groups, a column to a lane
    float pa = 1.f, ph = 0.f;
#pragma unroll
    for (int k = 0; k < GPW; ++k) {
        const float q = ga[w * GPW + k][lane];
        ph = pass<RESET>(q, gh[w * GPW + k][lane], ph);
        pa = join<RESET>(pa, q);
    }
    wa[w][lane] = pa;
    wh[w][lane] = ph;
    way.tell(next, &mine);
    __syncthreads();
    again(a);
    // wavefront 0 takes the chunk as a whole, a column to a lane: of the channel ch
    const int base = c0 + lane / V * V, ch = min(base, D - V) + lane % V;
    const bool there = base < D;
    const int64_t stride = (int64_t)a->cols * kCols, words = tile.b * a->nchunks * stride + c0;
    float ca = 1.f, chunk_h = 0.f;
    Entering<RESET> entering;
    if (w == 0 && a->nchunks > 1) {
#pragma unroll
        for (int k = 0; k < kGatedWaves; ++k) {
            chunk_h = pass<RESET>(wa[k][lane], wh[k][lane], chunk_h);
            ca = join<RESET>(ca, wa[k][lane]);
        }
        publish(a->pieces + words + tile.chunk * stride + lane, ca, chunk_h);
        entering.look(a->pieces + words, a->ends + words, stride, lane, tile.chunk);
    }
    way.go_on(a, &mine);
    if (w == 0) {
        float first = 0.f;
        if (a->init && there) first = a->init[tile.b * D + ch];
        if (a->nchunks > 1) {
            first = entering.state(a->pieces + words, a->ends + words, stride, lane, tile.chunk, first);
            publish(a->ends + words + tile.chunk * stride + lane, pass<RESET>(ca, chunk_h, first));
        }
        carry[lane] = first;
        if (a->states && there) a->states[(tile.b * a->nchunks + tile.chunk) * D + ch] = first;
    }
    __syncthreads();
    float s = carry[lane];
    for (int k = 0; k < w; ++k) s = pass<RESET>(wa[k][lane], wh[k][lane], s);
#pragma unroll
    for (int k = 0; k < GPW; ++k) {
        const float own = gh[w * GPW + k][lane];
        gh[w * GPW + k][lane] = s;
        s = pass<RESET>(ga[w * GPW + k][lane], own, s);
    }
    __builtin_amdgcn_wave_barrier();
    const Tokens<T> py(a->y, row0, D, g * R, d);
    open = ~0u;
    float from[V];
#pragma unroll
    for (int e = 0; e < V; ++e) from[e] = gh[g][j * V + e];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        open &= keep(r);
        const bool last = r < n && t0 + r == a->T - 1 && a->final;
        Packed<T, V> o;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float v = __builtin_fmaf(p[r][e], cut<RESET>(from[e], open), h[r][e]);
            if (last) a->final[tile.b * D + d + e] = v;
            o.set(e, v);
        }
        if (r < n) o.store(py.out(r));
    }
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
    const Decay g = decay_of<DECAY, true>(at<T>(a.f, b * a.ldf + d), DECAY == SSD_DECAY_RATE ? base2(a.rate[d]) : 0.f);
    float v = at<T>(a.x, b * a.ldx + d);
    if constexpr (IN) v *= sigmoid_of<true>(at<T>(a.i, b * a.ldi + d));
    h = g.a * h + g.c * v;
    a.state_out[k] = h;
    reinterpret_cast<T *>(a.y)[k] = (T)h;
}

GatedPlan gated_plan(int64_t batch, int64_t T, int64_t D, ssd_dtype dtype, bool backward) {
    GatedPlan p = {};
    p.cols = (D + kCols - 1) / kCols;
    p.nchunks = (T + SSD_GATED_CHUNK - 1) / SSD_GATED_CHUNK;
    const int64_t most = kMostThreads / kGatedThreads;  // one work-group for each
    p.fits = batch == 0 || T == 0 || (batch <= most / p.cols && batch * p.cols <= most / p.nchunks);
    if (!p.fits) return p;
    p.tiles = batch * p.cols * p.nchunks;
    // Tiles of a ticket: two of neighbouring columns where a tile takes the memory no longer than a ticket takes (13 ns): the
    // forward pass's in 16 bits, of 48 or 64 KB (with one, and with two: 2048 x 1536 20.3 and 18.3 us, 4 x 2048 x 4096 75 and
    // 72, 16384 x 4096 without input gates 124 and 105). Those in fp32 and the gradients' are larger (4 x 2048 x 4096 in fp32 107 and
    // 114, gradients in bf16 143 and 151), and below 384 tiles two in a row take a chunk longer than the tickets of two (2 x 8192 x
    // 64 18 and 22). Never of two chunks: a ticket that ended one and began the next would have each chunk wait for a second tile
    // of the one before.
    p.share = p.nchunks > 1 && !backward && dtype == SSD_BF16 && p.tiles >= 384 ? 2 : 1;
    const int64_t tickets = (batch * p.cols + p.share - 1) / p.share * p.nchunks;
    p.groups = p.nchunks > 1 && tickets > 768 ? 768 : tickets;  // 3 for each CU
    // the ticket, then a chunk's (a, h) and its end for each column
    p.word_bytes = p.nchunks > 1 && p.tiles ? 256 + p.tiles * kCols * 12 : 0;
    p.rate_bytes = batch * p.nchunks * D * 4;
    return p;
}

ssd_status clear_words(GatedArgs &a, const GatedPlan &p, void *workspace, hipStream_t s) {
    a.cols = (int)p.cols;
    a.share = (uint32_t)p.share;
    a.wide = (uint32_t)(a.batch * p.cols);
    a.tickets = (uint32_t)((a.batch * p.cols + p.share - 1) / p.share);
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
    return pick_gated(dtype, decay, a.i != nullptr, a.reset != nullptr, [&](auto t, auto dec, auto in, auto reset) {
        using T = decltype(t);
        constexpr int DECAY = decltype(dec)::value, V = 16 / (int)sizeof(T);
        constexpr bool IN = decltype(in)::value, RESET = decltype(reset)::value;
        auto go = [&](auto k) { return status_of(launch(k, dim3((unsigned)p.groups), dim3(kGatedThreads), s, a)); };
        return a.D >= V ? go(k_gated_fwd<T, DECAY, IN, RESET, V>) : go(k_gated_fwd<T, DECAY, IN, RESET, 1>);
    });
}

ssd_status launch_gated_step(const GatedStepArgs &a, ssd_dtype dtype, int decay, hipStream_t s) {
    return pick_gated(dtype, decay, a.i != nullptr, false, [&](auto t, auto dec, auto in, auto) {
        return status_of(launch(k_gated_step<decltype(t), decltype(dec)::value, decltype(in)::value>,
                                dim3((unsigned)((a.rows * a.D + kThreads - 1) / kThreads)), dim3(kThreads), s, a));
    });
}

}  // namespace ssd
