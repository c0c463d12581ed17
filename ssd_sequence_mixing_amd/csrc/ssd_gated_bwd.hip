// Gradients of the gated linear recurrence (ssd_gated.hip) for gfx950. With
// g_t = dy_t + G_{t+1}, where G_t = a_t g_t is what a token hands back to the one before:
//
//   dx = g c sigmoid(i);   di = g c x sigmoid(i) sigmoid(-i)
//   d log a = g (a h_{t-1} + v dc/d log a);   df = d log a dlog a/df;   drate = sum of d log a sigmoid(f)
//
// One pass over the inputs, from the last chunk to the first. The states that entered each chunk are
// given, so h is local to the chunk; G is handed on between chunks as the forward pass hands h on.
// A lane keeps its tokens as stored, with a and c; both walks over them are done
// twice, for the group's ends and from its entering values, which costs fewer registers than keeping them.
#include "ssd_gated.h"

namespace ssd {

template <typename T, int DECAY, bool IN, int V>
__global__ __launch_bounds__(kGatedThreads, 4) void k_gated_bwd(GatedArgs a) {
    using S = Shape<T, V>;
    constexpr int R = S::R, LPR = S::LPR, GPW = S::GPW;
    constexpr bool kFine = sizeof(T) == 4, kRate = DECAY == SSD_DECAY_RATE;
    // the groups' decays, ends of h and of G; then the values that enter them
    __shared__ __attribute__((aligned(16))) float ga[S::G][kCols], gh[S::G][kCols], gg[S::G][kCols];
    __shared__ float wa[kGatedWaves][kCols], wh[kGatedWaves][kCols], wg[kGatedWaves][kCols], carry[kCols];
    const Tile tile = take_tile(a.ticket, a.batch, a.cols);
    const int chunk = (int)a.nchunks - 1 - tile.chunk;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int j = lane % LPR, g = w * GPW + lane / LPR;
    const int D = (int)a.D, c0 = tile.col * kCols;
    const bool live = c0 + j * V < D;
    const int d = min(c0 + j * V, D - V);
    const int t0 = chunk * SSD_GATED_CHUNK + g * R;
    const int n = live ? min(R, (int)a.T - t0) : 0;
    const int64_t row = tile.b * a.T + t0;
    // the channel of this lane's column
    const int base = c0 + lane / V * V, ch = min(base, D - V) + lane % V;
    const bool there = base < D;

    Packed<T, V> x[R], f[R], in[IN ? R : 1], dy[R];
    uint32_t keep[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        x[r] = {}; f[r] = {}; dy[r] = {};
        if constexpr (IN) in[r] = {};
        keep[r] = ~0u;
        if (r < n) {
            f[r].load(reinterpret_cast<const T *>(a.f) + (row + r) * a.ldf + d);
            x[r].load(reinterpret_cast<const T *>(a.x) + (row + r) * a.ldx + d);
            if constexpr (IN) in[r].load(reinterpret_cast<const T *>(a.i) + (row + r) * a.ldi + d);
            dy[r].load(reinterpret_cast<const T *>(a.dy) + (row + r) * D + d);
        }
    }
    float enter = 0.f;  // the state before the chunk, of this lane's column
    if (there) enter = a.states[(tile.b * a.nchunks + chunk) * D + ch];
    if (a.reset) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (r < n && a.reset[row + r]) keep[r] = 0u;
    }
    float rate[V];
#pragma unroll
    for (int e = 0; e < V; ++e) rate[e] = kRate && live ? a.rate[d + e] : 0.f;

    float dec[R][V], c[R][V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float h = 0.f, p = 1.f, back = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const Decay q = decay_of<DECAY, kFine, false>(f[r].get(e), rate[e]);
            float v = x[r].get(e);
            if constexpr (IN) v *= sigmoid_of<kFine>(in[r].get(e));
            // tokens behind the end pass both on
            dec[r][e] = r < n ? q.a : 1.f;
            c[r][e] = r < n ? q.c : 0.f;
            h = __builtin_fmaf(dec[r][e], masked(h, keep[r]), c[r][e] * v);
            p = masked(p * dec[r][e], keep[r]);
        }
#pragma unroll
        for (int r = R - 1; r >= 0; --r) back = masked(dec[r][e] * (dy[r].get(e) + back), keep[r]);
        ga[g][j * V + e] = p;
        gh[g][j * V + e] = h;
        gg[g][j * V + e] = back;
    }
    __builtin_amdgcn_wave_barrier();
    // this wavefront's groups, a column to a lane
    float pa = 1.f, ph = 0.f, pg = 0.f;
#pragma unroll
    for (int k = 0; k < GPW; ++k) {
        const float q = ga[w * GPW + k][lane];
        ph = pass(q, gh[w * GPW + k][lane], ph);
        pa *= q;
    }
#pragma unroll
    for (int k = GPW - 1; k >= 0; --k) pg = pass(ga[w * GPW + k][lane], gg[w * GPW + k][lane], pg);
    wa[w][lane] = pa;
    wh[w][lane] = ph;
    wg[w][lane] = pg;
    __syncthreads();
    if (w == 0) {
        const int64_t at = tile.b * D + ch;
        float first = 0.f, ca = 1.f, cg = 0.f;
        if (a.dfinal && there) first = a.dfinal[at];
#pragma unroll
        for (int k = kGatedWaves - 1; k >= 0; --k) {
            cg = pass(wa[k][lane], wg[k][lane], cg);
            ca *= wa[k][lane];
        }
        if (a.nchunks > 1) {
            const int64_t stride = (int64_t)a.cols * kCols;
            uint64_t *pieces = a.pieces + tile.b * a.nchunks * stride + c0 + lane;
            uint32_t *ends = a.ends + tile.b * a.nchunks * stride + c0 + lane;
            const int k = tile.chunk;
            publish(pieces + k * stride, ca, cg);
            first = entering(pieces, ends, stride, k, first);
            publish(ends + k * stride, pass(ca, cg, first));
        }
        carry[lane] = first;
        if (chunk == 0 && a.dinit && there) a.dinit[at] = pass(ca, cg, first);
    }
    // the states that enter this wavefront's groups
    for (int k = 0; k < w; ++k) enter = pass(wa[k][lane], wh[k][lane], enter);
#pragma unroll
    for (int k = 0; k < GPW; ++k) {
        const float own = gh[w * GPW + k][lane];
        gh[w * GPW + k][lane] = enter;
        enter = pass(ga[w * GPW + k][lane], own, enter);
    }
    __syncthreads();
    float back = carry[lane];
    for (int k = kGatedWaves - 1; k > w; --k) back = pass(wa[k][lane], wg[k][lane], back);
#pragma unroll
    for (int k = GPW - 1; k >= 0; --k) {
        const float own = gg[w * GPW + k][lane];
        gg[w * GPW + k][lane] = back;
        back = pass(ga[w * GPW + k][lane], own, back);
    }
    __builtin_amdgcn_wave_barrier();

#pragma unroll
    for (int r = 0; r < R; ++r) {
        f[r].forget();
        if constexpr (IN) in[r].forget();
    }
    float before[R][V], later[V], sum[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        sum[e] = 0.f;
        later[e] = gg[g][j * V + e];
        before[0][e] = masked(gh[g][j * V + e], keep[0]);
#pragma unroll
        for (int r = 1; r < R; ++r) {
            float v = x[r - 1].get(e);
            if constexpr (IN) v *= sigmoid_of<kFine>(in[r - 1].get(e));
            before[r][e] = masked(__builtin_fmaf(dec[r - 1][e], before[r - 1][e], c[r - 1][e] * v), keep[r]);
        }
    }
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
        float dx[V], di[V], df[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float dh = dy[r].get(e) + later[e], xv = x[r].get(e), cc = c[r][e], aa = dec[r][e];
            later[e] = masked(aa * dh, keep[r]);
            Gate gi = {1.f, 0.f};
            if constexpr (IN) gi = gate_of<kFine>(in[r].get(e));
            const float v = xv * gi.s, u = dh * cc;
            dx[e] = u * gi.s;
            di[e] = u * v * gi.n;
            float dla = aa * before[r][e];
            if constexpr (DECAY == SSD_DECAY_LOG) {
                dla *= dh;
                df[e] = dla;
            } else if constexpr (DECAY == SSD_DECAY_SIGMOID) {  // c = sigmoid(-f)
                dla = dh * __builtin_fmaf(-aa, v, dla);
                df[e] = dla * cc;
            } else {
                // dc / d log a = -a^2 / c; none where c is 0
                const float slope = cc > 0.f ? -aa * aa * __builtin_amdgcn_rcpf(cc) : 0.f;
                dla = dh * __builtin_fmaf(slope, v, dla);
                const Gate q = gate_of<kFine>(f[r].get(e));
                const float by = dla * q.s;
                df[e] = by * q.n * rate[e];
                sum[e] += r < n ? by : 0.f;
            }
        }
        if (r < n) {
            const int64_t at = (row + r) * D + d;
            Packed<T, V>::store(reinterpret_cast<T *>(a.dx) + at, dx);
            if constexpr (IN) Packed<T, V>::store(reinterpret_cast<T *>(a.di) + at, di);
            Packed<T, V>::store(reinterpret_cast<T *>(a.df) + at, df);
        }
    }
    if constexpr (kRate) {
#pragma unroll
        for (int e = 0; e < V; ++e) ga[g][j * V + e] = sum[e];  // read so far by this wavefront alone
        __builtin_amdgcn_wave_barrier();
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < GPW; ++k) s += ga[w * GPW + k][lane];
        __syncthreads();  // wa has been read
        wa[w][lane] = s;
        __syncthreads();
        if (w == 0 && there) {
            s = wa[0][lane];
#pragma unroll
            for (int k = 1; k < kGatedWaves; ++k) s += wa[k][lane];
            a.part[(tile.b * a.nchunks + chunk) * D + ch] = s;
        }
    }
}

ssd_status launch_gated_bwd(GatedArgs a, const GatedPlan &p, ssd_dtype dtype, int decay, void *workspace, hipStream_t s) {
    ssd_status st = clear_words(a, p, workspace, s);
    if (st != SSD_OK) return st;
    a.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + p.word_bytes);
    st = pick_gated(dtype, decay, a.i != nullptr, [&](auto t, auto dec, auto in) {
        using T = decltype(t);
        constexpr int DECAY = decltype(dec)::value, V = 16 / (int)sizeof(T);
        constexpr bool IN = decltype(in)::value;
        auto go = [&](auto k) { return status_of(launch(k, dim3((unsigned)p.tiles), dim3(kGatedThreads), s, a)); };
        return a.D >= V ? go(k_gated_bwd<T, DECAY, IN, V>) : go(k_gated_bwd<T, DECAY, IN, 1>);
    });
    if (st != SSD_OK || !a.drate) return st;
    return launch_column_sums(a.part, a.drate, (int)(a.batch * a.nchunks), a.D, s);
}

}  // namespace ssd
