// One recurrent decode step for gfx950: the O(1)-per-token inference form of
// the SSM ("Transformer vs Mamba/SSM: the next step of the architecture",
// why it matters: each step only updates a fixed-size state).
//
//   a = exp(dt[b,h] A[h]);  s[p,n] <- a s[p,n] + dt x[p] B[g,n];
//   y[p] = sum_n s[p,n] C[g,n] + D[h] x[p]
//
// from the state of row parent[b] (kBeam: beam search's reordering of states,
// which costs no pass of its own) or of row b in place, and
// optionally with the layer's prologue and epilogue fused in: dt =
// softplus(dt + dt_bias[h]), the input x <- SiLU(b + w . [x_{t-3}, x_{t-2},
// x_{t-1}, x_t]) of the layer's causal convolution (the 3 earlier raw inputs
// kept in a rolling conv state, shifted by this step) and y <- y * silu(z[p]).
//
// The state is the only large operand: the kernel streams it once in and
// once out with 16-byte non-temporal accesses (it is not reused by this
// step, so it should not displace anything in the caches). A row of N fp32
// values is split over N/4 lanes; the dot product with C is reduced across
// those lanes with cross-lane shuffles. Each work-group covers RPB rows of
// one (batch, head), so the head's scalars (dt, A, D, group) are uniform
// and every lane keeps two rows' loads in flight.
// From parents' rows the states' addresses wait for one scalar load more: 32
// sequences of 8 beams, 64 heads of 64 x 128: 176 us (0.54 GB written, and 0.35 GB read where random parents are
// two thirds of the rows; in place 0.54 GB each way take 181).
#include "ssd_common.h"
#include "ssd_internal.h"

namespace ssd {

constexpr int kStepThreads = 256;
constexpr int kStepUnroll = 2;

template <typename TI, int N>
struct StepShape {
    static constexpr int TPR = N / 4;                 // lanes per state row
    static constexpr int RPW = 64 / TPR;              // rows per wavefront per pass
    static constexpr int RPB = (kStepThreads / 64) * RPW * kStepUnroll;  // rows per work-group
};

template <typename TI, int N, bool kBeam>
__global__ __launch_bounds__(kStepThreads) void k_step(StepArgs a, int pblocks) {
    using Tr = Traits<TI>;
    using S = StepShape<TI, N>;
    constexpr int TPR = S::TPR, RPW = S::RPW, RPB = S::RPB;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int sub = lane / TPR, c4 = lane % TPR;
    const int P = (int)a.P, H = (int)a.H, G = (int)a.G;
    // work-group -> (batch*head, block of rows); all of it scalar
    const int64_t bh = blockIdx.x / pblocks;
    const int pb = blockIdx.x - (int)(bh * pblocks);
    const int64_t bb = bh / H;
    const int h = (int)(bh - bb * H);
    const int g = (h * G) / H;
    float dtv = Tr::to_f32(reinterpret_cast<const TI *>(a.dt)[bh]);
    if (a.dt_bias || a.softplus) dtv = dt_prologue(dtv, a.dt_bias ? a.dt_bias[h] : 0.f, a.softplus);
    const float dec = fast_exp2(dtv * a.A[h] * kLog2e);
    const float Dh = a.D[h];
    float *srow = a.state + bh * P * N;
    // kBeam: the row the state comes from; out of range, a sequence that begins
    // (zero state). The states' addresses then wait for this one scalar load.
    int64_t from = bb;
    bool begun = true;
    const float *sin = srow;
    if constexpr (kBeam) {
        from = a.parent[bb];
        begun = from >= 0 && from < a.src_rows;
        if (!begun) from = 0;
        sin = a.state_in + (from * H + h) * P * N;
    }

    int p[kStepUnroll];
    f32x4 s[kStepUnroll];
#pragma unroll
    for (int u = 0; u < kStepUnroll; ++u) {
        p[u] = pb * RPB + (u * (kStepThreads / 64) + w) * RPW + sub;
        s[u] = (p[u] < P && begun)
                   ? __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(sin + (int64_t)p[u] * N) + c4)
                   : f32x4{0.f, 0.f, 0.f, 0.f};
    }
    const TI *bp = reinterpret_cast<const TI *>(a.B) + (bb * G + g) * N + 4 * c4;
    const TI *cp = reinterpret_cast<const TI *>(a.C) + (bb * G + g) * N + 4 * c4;
    float bv[4], cv[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        bv[e] = Tr::to_f32(bp[e]);
        cv[e] = Tr::to_f32(cp[e]);
    }
#pragma unroll
    for (int u = 0; u < kStepUnroll; ++u) {
        const bool ok = p[u] < P;
        float xv = ok ? Tr::to_f32(reinterpret_cast<const TI *>(a.x)[bh * P + p[u]]) : 0.f;
        if (a.conv_w && ok) {
            // channel c = h P + p: x' = SiLU(b + w0 s0 + w1 s1 + w2 s2 + w3 x), in fp32 and
            // rounded to the storage type (as the forward stages it); the conv
            // state then holds (s1, s2, x). Every lane of the row reads it, one writes it,
            // after the reads have been used.
            const int64_t ch = (int64_t)h * P + p[u];
            TI *cst = reinterpret_cast<TI *>(a.conv_state) + (bb * H * P + ch) * 3;
            const TI *old = cst;
            if constexpr (kBeam) old = reinterpret_cast<const TI *>(a.conv_in) + (from * H * P + ch) * 3;
            const TI s1 = begun ? old[1] : Tr::from_f32(0.f), s2 = begun ? old[2] : Tr::from_f32(0.f);
            const float s0 = begun ? Tr::to_f32(old[0]) : 0.f;
            const f32x4 wv = *reinterpret_cast<const f32x4 *>(a.conv_w + 4 * ch);
            const float v = (a.conv_b ? a.conv_b[ch] : 0.f) + wv[0] * s0 + wv[1] * Tr::to_f32(s1) +
                            wv[2] * Tr::to_f32(s2) + wv[3] * xv;
            const float xa = Tr::to_f32(Tr::from_f32(v / (1.f + expf(-v))));
            if (c4 == 0) {
                cst[0] = s1;
                cst[1] = s2;
                cst[2] = Tr::from_f32(xv);
            }
            xv = xa;
        }
        const float uin = dtv * xv;
        f32x4 sn;
        float part = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sn[e] = dec * s[u][e] + uin * bv[e];
            part += sn[e] * cv[e];
        }
        if (ok) __builtin_nontemporal_store(sn, reinterpret_cast<f32x4 *>(srow + (int64_t)p[u] * N) + c4);
#pragma unroll
        for (int off = TPR / 2; off > 0; off >>= 1) part += __shfl_xor(part, off, 64);
        if (ok && c4 == 0) {
            float yv = part + Dh * xv;
            if (a.z) yv = silu_gate(yv, Tr::to_f32(reinterpret_cast<const TI *>(a.z)[bh * P + p[u]]));
            reinterpret_cast<TI *>(a.y)[bh * P + p[u]] = Tr::from_f32(yv);
        }
    }
}

// Rows b0 .. b0 + n - 1 of a step (the rows that they come from stay what they are).
template <typename TI>
static StepArgs step_rows(const StepArgs &a, int64_t b0, int64_t n) {
    StepArgs r = a;
    const int64_t hp = a.H * a.P;
    r.batch = n;
    r.state += b0 * hp * a.N;
    r.x = static_cast<const TI *>(a.x) + b0 * hp;
    r.dt = static_cast<const TI *>(a.dt) + b0 * a.H;
    r.B = static_cast<const TI *>(a.B) + b0 * a.G * a.N;
    r.C = static_cast<const TI *>(a.C) + b0 * a.G * a.N;
    r.y = static_cast<TI *>(a.y) + b0 * hp;
    if (a.z) r.z = static_cast<const TI *>(a.z) + b0 * hp;
    if (a.conv_w) r.conv_state = static_cast<TI *>(a.conv_state) + b0 * hp * 3;
    if (a.parent) r.parent += b0;
    return r;
}

template <typename TI, int N, bool kBeam>
static ssd_status run_step(const StepArgs &a, hipStream_t s) {
    constexpr int RPB = StepShape<TI, N>::RPB;
    const int pblocks = (int)((a.P + RPB - 1) / RPB);
    // as many rows as one launch takes, and the rest in more
    const int64_t most = kMostThreads / kStepThreads / (a.H * pblocks);
    if (most == 0) return SSD_ERR_UNSUPPORTED;
    for (int64_t b0 = 0; b0 < a.batch; b0 += most) {
        const int64_t n = a.batch - b0 < most ? a.batch - b0 : most;
        if (launch(k_step<TI, N, kBeam>, dim3((unsigned)(n * a.H * pblocks)), dim3(kStepThreads), s,
                   step_rows<TI>(a, b0, n), pblocks) != hipSuccess)
            return SSD_ERR_HIP;
    }
    return SSD_OK;
}

template <typename TI, bool kBeam>
static ssd_status step_n(const StepArgs &a, hipStream_t s) {
    switch (a.N) {
        case 4: return run_step<TI, 4, kBeam>(a, s);
        case 8: return run_step<TI, 8, kBeam>(a, s);
        case 16: return run_step<TI, 16, kBeam>(a, s);
        case 32: return run_step<TI, 32, kBeam>(a, s);
        case 64: return run_step<TI, 64, kBeam>(a, s);
        case 128: return run_step<TI, 128, kBeam>(a, s);
        case 256: return run_step<TI, 256, kBeam>(a, s);
        default: return SSD_ERR_UNSUPPORTED;
    }
}

ssd_status launch_step(const StepArgs &a, hipStream_t s) {
    if (a.parent) return a.dtype == SSD_BF16 ? step_n<bf16, true>(a, s) : step_n<float, true>(a, s);
    return a.dtype == SSD_BF16 ? step_n<bf16, false>(a, s) : step_n<float, false>(a, s);
}

}  // namespace ssd
