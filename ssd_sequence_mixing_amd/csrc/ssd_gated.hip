// Gated linear recurrence for gfx950: per channel d of a sequence
//
//   h_t = a_t h_{t-1} + c_t v_t,   v_t = sigmoid(i_t) x_t,   y_t = h_t
//
// with the decay a_t in (0, 1] and the input's coefficient c_t made from a
// gate f_t: log a = f, c = 1; or a = sigmoid(f), c = 1 - a; or
// log a = rate[d] sigmoid(f), c = sqrt(1 - a^2). reset[t] leaves out h_{t-1}.
#include <type_traits>

#include "ssd_common.h"
#include "ssd_internal.h"

namespace ssd {

constexpr int kThreads = 256;

// e^x within 2^-22 of itself: x log2 e in two parts, since the rounding of the first
// is 2^-24 of it, some 1e-6 of the result far from zero. 0 and infinity beyond 200.
__device__ __forceinline__ float exp_of(float x) {
    x = x < -200.f ? -200.f : x;
    x = x > 200.f ? 200.f : x;
    const float y = x * kLog2e, rest = __builtin_fmaf(x, kLog2e, -y) + x * 1.925963033e-8f;
    const float e = fast_exp2(y);
    return __builtin_fmaf(e * kLn2, rest, e);
}

// sigmoid(v) and sigmoid(-v), both to a few 2^-24 of themselves.
struct Gate {
    float s, n;
};
__device__ __forceinline__ Gate gate_of(float v) {
    const float e = exp_of(-fabsf(v)), r = __builtin_amdgcn_rcpf(1.f + e), er = e * r;
    return v < 0.f ? Gate{er, r} : Gate{r, er};
}

// The decay and the input's coefficient of one token's gate; and what the
// gradients take: slope = d c / d log a, p = d log a / d f, s = sigmoid(f).
struct Decay {
    float a, c, slope, p, s;
};
// 1 - e^z for z <= 0: near zero by its series (8 terms: 2^-27 of it at z = -1/2), where the difference would cancel.
__device__ __forceinline__ float one_minus_exp(float z, float e) {
    const float q = 1.f + z * (1 / 2.f) * (1.f + z * (1 / 3.f) * (1.f + z * (1 / 4.f) * (1.f + z * (1 / 5.f) * (1.f + z * (1 / 6.f) * (1.f + z * (1 / 7.f) * (1.f + z * (1 / 8.f)))))));
    return z > -0.5f ? -z * q : 1.f - e;
}
template <int DECAY>
__device__ __forceinline__ Decay decay_of(float f, float rate) {
    Decay o;
    if constexpr (DECAY == SSD_DECAY_LOG) {
        o.a = exp_of(f);
        o.c = 1.f; o.slope = 0.f; o.p = 1.f; o.s = 0.f;
    } else if constexpr (DECAY == SSD_DECAY_SIGMOID) {
        const Gate g = gate_of(f);
        o.a = g.s; o.c = g.n; o.slope = -g.s; o.p = g.n; o.s = 0.f;
    } else {
        const Gate g = gate_of(f);
        const float la = rate * g.s;
        o.a = exp_of(la);
        const float a2 = o.a * o.a, c2 = one_minus_exp(2.f * la, a2);
        // a decay of 1 (and above: a positive rate) takes no input, and has no slope
        const float r = c2 < 0x1p-100f ? 0.f : __builtin_amdgcn_rsqf(c2);
        o.c = c2 * r; o.slope = -a2 * r; o.p = la * g.n; o.s = g.s;
    }
    return o;
}

template <typename T>
__device__ __forceinline__ float at(const void *p, int64_t i) {
    return (float)reinterpret_cast<const T *>(p)[i];
}

template <typename T, int DECAY, bool IN>
__global__ __launch_bounds__(kThreads) void k_gated_fwd(GatedArgs a) {
    const int64_t k = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (k >= a.batch * a.D) return;
    const int64_t b = k / a.D, d = k - b * a.D;
    const float rate = DECAY == SSD_DECAY_RATE ? a.rate[d] : 0.f;
    float h = a.init ? a.init[k] : 0.f;
    for (int64_t t = 0; t < a.T; ++t) {
        const int64_t row = b * a.T + t;
        if (a.states && t % SSD_GATED_CHUNK == 0) a.states[(b * a.nchunks + t / SSD_GATED_CHUNK) * a.D + d] = h;
        const Decay g = decay_of<DECAY>(at<T>(a.f, row * a.ldf + d), rate);
        float v = at<T>(a.x, row * a.ldx + d);
        if constexpr (IN) v *= gate_of(at<T>(a.i, row * a.ldi + d)).s;
        const bool cut = a.reset && a.reset[row];
        h = (cut ? 0.f : g.a * h) + g.c * v;
        reinterpret_cast<T *>(a.y)[row * a.D + d] = (T)h;
    }
    if (a.final) a.final[k] = h;
}

template <typename T, int DECAY, bool IN>
__global__ __launch_bounds__(kThreads) void k_gated_bwd(GatedArgs a) {
    const int64_t k = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (k >= a.batch * a.D) return;
    const int64_t b = k / a.D, d = k - b * a.D;
    const float rate = DECAY == SSD_DECAY_RATE ? a.rate[d] : 0.f;
    float back = a.dfinal ? a.dfinal[k] : 0.f, drate = 0.f;
    float before[SSD_GATED_CHUNK];
    for (int64_t c = a.nchunks - 1; c >= 0; --c) {
        float h = a.states[(b * a.nchunks + c) * a.D + d];
        const int64_t t0 = c * SSD_GATED_CHUNK, n = a.T - t0 < SSD_GATED_CHUNK ? a.T - t0 : SSD_GATED_CHUNK;
        for (int pass = 0; pass < 2; ++pass)
            for (int64_t j = 0; j < n; ++j) {
                const int64_t row = b * a.T + t0 + (pass ? n - 1 - j : j);
                const Decay g = decay_of<DECAY>(at<T>(a.f, row * a.ldf + d), rate);
                const float x = at<T>(a.x, row * a.ldx + d);
                Gate in = {1.f, 0.f};
                if constexpr (IN) in = gate_of(at<T>(a.i, row * a.ldi + d));
                const float v = x * in.s;
                const bool cut = a.reset && a.reset[row];  // what lies before may be infinite or NaN: left out, not multiplied by 0
                if (!pass) {
                    before[j] = cut ? 0.f : h;
                    h = (cut ? 0.f : g.a * h) + g.c * v;
                } else {
                    const float dh = at<T>(a.dy, row * a.D + d) + back;
                    back = cut ? 0.f : g.a * dh;
                    const float dla = back * before[n - 1 - j] + dh * g.slope * v;
                    reinterpret_cast<T *>(a.dx)[row * a.D + d] = (T)(dh * g.c * in.s);
                    if constexpr (IN) reinterpret_cast<T *>(a.di)[row * a.D + d] = (T)(dh * g.c * v * in.n);
                    reinterpret_cast<T *>(a.df)[row * a.D + d] = (T)(dla * g.p);
                    drate += dla * g.s;
                }
            }
    }
    if (a.dinit) a.dinit[k] = back;
    if (DECAY == SSD_DECAY_RATE && a.part) a.part[k] = drate;
}

template <typename T, int DECAY, bool IN>
__global__ __launch_bounds__(kThreads) void k_gated_step(GatedStepArgs a) {
    const int64_t k = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (k >= a.rows * a.D) return;
    const int64_t b = k / a.D, d = k - b * a.D;
    const int64_t from = a.parent ? a.parent[b] : b;
    float h = from >= 0 && from < a.src ? a.state_in[from * a.D + d] : 0.f;
    const Decay g = decay_of<DECAY>(at<T>(a.f, b * a.ldf + d), DECAY == SSD_DECAY_RATE ? a.rate[d] : 0.f);
    float v = at<T>(a.x, b * a.ldx + d);
    if constexpr (IN) v *= gate_of(at<T>(a.i, b * a.ldi + d)).s;
    h = g.a * h + g.c * v;
    a.state_out[k] = h;
    reinterpret_cast<T *>(a.y)[k] = (T)h;
}

// fn(types...) for the call's storage type, decay and whether the input is gated.
template <typename F>
static ssd_status pick(ssd_dtype dtype, int decay, bool in, F fn) {
    auto two = [&](auto t, auto dec) {
        return in ? fn(t, dec, std::true_type{}) : fn(t, dec, std::false_type{});
    };
    auto one = [&](auto t) {
        if (decay == SSD_DECAY_LOG) return two(t, std::integral_constant<int, SSD_DECAY_LOG>{});
        if (decay == SSD_DECAY_SIGMOID) return two(t, std::integral_constant<int, SSD_DECAY_SIGMOID>{});
        return two(t, std::integral_constant<int, SSD_DECAY_RATE>{});
    };
    return dtype == SSD_BF16 ? one(bf16{}) : one(float{});
}
static ssd_status status_of(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

GatedPlan gated_plan(int64_t batch, int64_t T, int64_t D, ssd_dtype) {
    GatedPlan p = {};
    p.fits = true;
    p.rate_bytes = (batch * D * 4 + 255) & ~(int64_t)255;
    return p;
}

ssd_status launch_gated_fwd(GatedArgs a, const GatedPlan &, ssd_dtype dtype, int decay, void *, hipStream_t s) {
    return pick(dtype, decay, a.i != nullptr, [&](auto t, auto dec, auto in) {
        return status_of(launch(k_gated_fwd<decltype(t), decltype(dec)::value, decltype(in)::value>,
                                dim3((unsigned)((a.batch * a.D + kThreads - 1) / kThreads)), dim3(kThreads), s, a));
    });
}

ssd_status launch_gated_bwd(GatedArgs a, const GatedPlan &, ssd_dtype dtype, int decay, void *workspace, hipStream_t s) {
    a.part = static_cast<float *>(workspace);
    const ssd_status st = pick(dtype, decay, a.i != nullptr, [&](auto t, auto dec, auto in) {
        return status_of(launch(k_gated_bwd<decltype(t), decltype(dec)::value, decltype(in)::value>,
                                dim3((unsigned)((a.batch * a.D + kThreads - 1) / kThreads)), dim3(kThreads), s, a));
    });
    if (st != SSD_OK || !a.drate) return st;
    return launch_column_sums(a.part, a.drate, (int)a.batch, a.D, s);
}

ssd_status launch_gated_step(const GatedStepArgs &a, ssd_dtype dtype, int decay, hipStream_t s) {
    return pick(dtype, decay, a.i != nullptr, [&](auto t, auto dec, auto in) {
        return status_of(launch(k_gated_step<decltype(t), decltype(dec)::value, decltype(in)::value>,
                                dim3((unsigned)((a.rows * a.D + kThreads - 1) / kThreads)), dim3(kThreads), s, a));
    });
}

}  // namespace ssd
