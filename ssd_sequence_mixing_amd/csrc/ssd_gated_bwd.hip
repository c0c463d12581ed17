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

template <int N>
__device__ __forceinline__ void put(float *p, const float (&v)[N]) {
    if constexpr (N == 4) *reinterpret_cast<f32x4 *>(p) = f32x4{v[0], v[1], v[2], v[3]};
    else p[0] = v[0];
}
template <int N>
__device__ __forceinline__ void get(const float *p, float (&v)[N]) {
    if constexpr (N == 4) {
        const f32x4 q = *reinterpret_cast<const f32x4 *>(p);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = q[k];
    } else {
        v[0] = p[0];
    }
}

// What bounds it: the vector unit is busy 61% of the time (some 85 operations a value, 11 of them transcendental) and
// the registers leave 2 work-groups a CU, so that a tile's loads, walks and exchanges overlap little. In fp32 with input gates, decays
// from sigmoids or rates leave 1 (140 to 152 registers). 8 x 2048 x 1536 in bf16, rates
// and input gates (353 MB): 115 us, 119 with the words' clearing and the rates' sums (3.0 TB/s); in fp32 177. No kernel here spills
// vector registers: with 18 to 60 of them spilled it took 170 to 190. (V = 1 spills 14 to 68 scalar ones.)
template <typename T, int DECAY, bool IN, bool RESET, int V>
__global__ __launch_bounds__(kGatedThreads, V > 1 && (sizeof(T) == 2 || !IN) ? 4 : 2) void k_gated_bwd(GatedArgs) {
    Args a = args();
    using S = Shape<T, V>;
    constexpr int R = S::R, LPR = S::LPR, GPW = S::GPW;
    constexpr bool kFine = sizeof(T) == 4, kRate = DECAY == SSD_DECAY_RATE;
    // the groups' decays, ends of h and of G; then the values that enter them
    __shared__ __attribute__((aligned(16))) float ga[S::G][kCols], gh[S::G][kCols], gg[S::G][kCols];
    // by turns, since a wavefront that is done with a tile writes the next one's while others still read
    __shared__ float wa2[2][kGatedWaves][kCols], wh2[2][kGatedWaves][kCols], wg2[2][kGatedWaves][kCols], carry2[2][kCols];
    __shared__ uint32_t mine;
    Way way(a, &mine);
    for (uint32_t turn = 0; way.chunk < a->nchunks; ++turn) {
    again(a);
    const Tile tile = way.tile((uint32_t)a->cols);
    auto &wa = wa2[turn & 1], &wh = wh2[turn & 1], &wg = wg2[turn & 1];
    auto &carry = carry2[turn & 1];
    const int chunk = (int)a->nchunks - 1 - tile.chunk;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int j = lane % LPR, g = w * GPW + lane / LPR;
    const int D = (int)a->D, c0 = tile.col * kCols;
    const bool live = c0 + j * V < D;
    const int d = min(c0 + j * V, D - V);
    const int t0 = chunk * SSD_GATED_CHUNK + g * R;
    const int n = live ? min(R, (int)a->T - t0) : 0;
    const int64_t row0 = tile.b * a->T + (int64_t)chunk * SSD_GATED_CHUNK;
    const Tokens<T> px(a->x, row0, a->ldx, g * R, d), pf(a->f, row0, a->ldf, g * R, d), pi(a->i, row0, a->ldi, g * R, d), py(a->dy, row0, D, g * R, d);
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
            f[r].load(pf[r]);
            x[r].load(px[r]);
            if constexpr (IN) in[r].load(pi[r]);
            dy[r].load(py[r]);
        }
    }
    float enter = 0.f;  // the state before the chunk, of this lane's column
    if (there) enter = a->states[(tile.b * a->nchunks + chunk) * D + ch];
    if constexpr (RESET) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (r < n && a->reset[row0 + g * R + r]) keep[r] = 0u;
    }
    // read where it is needed, twice, and not kept
    auto rate = [&](int e) { return kRate ? base2(a->rate[d + e]) : 0.f; };
    const uint32_t next = way.ask(a);
    float dec[R][V], c[R][V];
    constexpr int B = V < 4 ? V : 4;  // channels that go to LDS together: one by one, 8 lanes would meet in one bank
#pragma unroll
    for (int b = 0; b < V; b += B) {
        float ps[B], hs[B], backs[B];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const int e = b + k;
            const float rate2 = rate(e);
            float h = 0.f, p = 1.f, back = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const Decay q = passed<DECAY, RESET>(decay_of<DECAY, kFine>(f[r].get(e), rate2), keep[r]);
                float v = x[r].get(e);
                if constexpr (IN) v *= sigmoid_of<kFine>(in[r].get(e));
                // tokens behind the last one, with x and dy zero, hand G on as it is
                const float dec_r = r < n ? q.a : 1.f;
                dec[r][e] = dec_r;
                c[r][e] = q.c;
                h = r ? __builtin_fmaf(dec_r, cut<RESET>(h, keep[r]), q.c * v) : q.c * v;
                p = r ? p * dec_r : dec_r;
            }
#pragma unroll
            for (int r = R - 1; r >= 0; --r) back = cut<RESET>(dec[r][e] * (dy[r].get(e) + back), keep[r]);
            uint32_t open = keep[0];
#pragma unroll
            for (int r = 1; r < R; ++r) open &= keep[r];
            ps[k] = mark<RESET>(p, open);
            hs[k] = h;
            backs[k] = back;
            if (k & 1) __builtin_amdgcn_sched_barrier(0);
        }
        put<B>(&ga[g][j * V + b], ps);
        put<B>(&gh[g][j * V + b], hs);
        put<B>(&gg[g][j * V + b], backs);
    }
    __builtin_amdgcn_wave_barrier();
    // this wavefront's groups, a column to a lane
    float pa = 1.f, ph = 0.f, pg = 0.f;
#pragma unroll
    for (int k = 0; k < GPW; ++k) {
        const float q = ga[w * GPW + k][lane];
        ph = pass<RESET>(q, gh[w * GPW + k][lane], ph);
        pa = join<RESET>(pa, q);
    }
#pragma unroll
    for (int k = GPW - 1; k >= 0; --k) pg = pass<RESET>(ga[w * GPW + k][lane], gg[w * GPW + k][lane], pg);
    wa[w][lane] = pa;
    wh[w][lane] = ph;
    wg[w][lane] = pg;
    way.tell(next, &mine);
    __syncthreads();
    way.go_on(a, &mine);
    again(a);
    if (w == 0) {
        const int64_t at = tile.b * D + ch;
        float first = 0.f, ca = 1.f, cg = 0.f;
        if (a->dfinal && there) first = a->dfinal[at];
#pragma unroll
        for (int k = kGatedWaves - 1; k >= 0; --k) {
            cg = pass<RESET>(wa[k][lane], wg[k][lane], cg);
            ca = join<RESET>(ca, wa[k][lane]);
        }
        if (a->nchunks > 1) {
            const int64_t stride = (int64_t)a->cols * kCols, words = tile.b * a->nchunks * stride + c0;
            const int k = tile.chunk;
            publish(a->pieces + words + k * stride + lane, ca, cg);
            Entering<RESET> entering;
            entering.look(a->pieces + words, a->ends + words, stride, lane, k);
            first = entering.state(a->pieces + words, a->ends + words, stride, lane, k, first);
            publish(a->ends + words + k * stride + lane, pass<RESET>(ca, cg, first));
        }
        carry[lane] = first;
        if (chunk == 0 && a->dinit && there) a->dinit[at] = pass<RESET>(ca, cg, first);
    }
    // the states that enter this wavefront's groups
    for (int k = 0; k < w; ++k) enter = pass<RESET>(wa[k][lane], wh[k][lane], enter);
#pragma unroll
    for (int k = 0; k < GPW; ++k) {
        const float own = gh[w * GPW + k][lane];
        gh[w * GPW + k][lane] = enter;
        enter = pass<RESET>(ga[w * GPW + k][lane], own, enter);
    }
    __syncthreads();
    float back = carry[lane];
    for (int k = kGatedWaves - 1; k > w; --k) back = pass<RESET>(wa[k][lane], wg[k][lane], back);
#pragma unroll
    for (int k = GPW - 1; k >= 0; --k) {
        const float own = gg[w * GPW + k][lane];
        gg[w * GPW + k][lane] = back;
        back = pass<RESET>(ga[w * GPW + k][lane], own, back);
    }
    __builtin_amdgcn_wave_barrier();
    // ga is read for the last time above
#pragma unroll
    for (int r = 0; r < R; ++r) {
        x[r].forget();
        f[r].forget();
        if constexpr (IN) in[r].forget();
    }
    // channel by channel (in pairs, where two make a stored word), so that its inputs' registers become its outputs'
    Packed<T, V> dx[R], di[R], df[R];
#pragma unroll
    for (int b = 0; b < V; b += B) {
        float enters[B], returns[B], sums[B];
        get<B>(&gh[g][j * V + b], enters);
        get<B>(&gg[g][j * V + b], returns);
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const int e = b + k;
            Gate gi[R];
            float before[R], v[R], later = returns[k], sum = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                gi[r] = {1.f, 0.f};
                if constexpr (IN) gi[r] = gate_of<kFine>(in[r].get(e));
                v[r] = x[r].get(e) * gi[r].s;
                before[r] = cut<RESET>(r ? __builtin_fmaf(dec[r ? r - 1 : 0][e], before[r ? r - 1 : 0], c[r ? r - 1 : 0][e] * v[r ? r - 1 : 0]) : enters[k], keep[r]);
            }
            const float by_rate = rate(e) * kLn2;
#pragma unroll
            for (int r = R - 1; r >= 0; --r) {
                const float dh = dy[r].get(e) + later, cc = c[r][e], aa = dec[r][e], u = dh * cc;
                const float back_r = aa * dh;
                later = cut<RESET>(back_r, keep[r]);
                dx[r].set(e, u * gi[r].s);
                if constexpr (IN) di[r].set(e, u * v[r] * gi[r].n);
                if constexpr (DECAY == SSD_DECAY_LOG) {
                    df[r].set(e, back_r * before[r]);
                } else if constexpr (DECAY == SSD_DECAY_SIGMOID) {  // c = sigmoid(-f)
                    df[r].set(e, cc * back_r * (before[r] - v[r]));
                } else {
                    // dc / d log a = -a^2 / c; none where c is 0
                    const float inv = cc > 0.f ? __builtin_amdgcn_rcpf(cc) : 0.f;
                    const Gate q = gate_of<kFine>(f[r].get(e));
                    const float by = back_r * __builtin_fmaf(-aa * v[r], inv, before[r]) * q.s;
                    df[r].set(e, by * q.n * by_rate);
                    sum += r < n ? by : 0.f;
                }
            }
            sums[k] = sum;
            if (k & 1) __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (kRate) put<B>(&ga[g][j * V + b], sums);  // its decays have been read, by this wavefront alone
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (r < n) {
            dx[r].store(Tokens<T>(a->dx, row0, D, g * R, d).out(r));
            if constexpr (IN) di[r].store(Tokens<T>(a->di, row0, D, g * R, d).out(r));
            df[r].store(Tokens<T>(a->df, row0, D, g * R, d).out(r));
        }
    if constexpr (kRate) {
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
            a->part[(tile.b * a->nchunks + chunk) * D + ch] = s;
        }
    }
    }
}

ssd_status launch_gated_bwd(GatedArgs a, const GatedPlan &p, ssd_dtype dtype, int decay, void *workspace, hipStream_t s) {
    ssd_status st = clear_words(a, p, workspace, s);
    if (st != SSD_OK) return st;
    a.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + p.word_bytes);
    st = pick_gated(dtype, decay, a.i != nullptr, a.reset != nullptr, [&](auto t, auto dec, auto in, auto reset) {
        using T = decltype(t);
        constexpr int DECAY = decltype(dec)::value, V = 16 / (int)sizeof(T);
        constexpr bool IN = decltype(in)::value, RESET = decltype(reset)::value;
        const int64_t groups = p.nchunks > 1 && p.groups > 512 ? 512 : p.groups;  // 2 for each CU
        auto go = [&](auto k) { return status_of(launch(k, dim3((unsigned)groups), dim3(kGatedThreads), s, a)); };
        return a.D >= V ? go(k_gated_bwd<T, DECAY, IN, RESET, V>) : go(k_gated_bwd<T, DECAY, IN, RESET, 1>);
    });
    if (st != SSD_OK || !a.drate) return st;
    return launch_column_sums(a.part, a.drate, (int)(a.batch * a.nchunks), a.D, s);
}

}  // namespace ssd
