// The gated linear recurrence's decay and gates, and how its chunks hand their states on
// (ssd_gated.hip, ssd_gated_bwd.hip).
#pragma once

#include <type_traits>

#include "ssd_common.h"
#include "ssd_internal.h"

namespace ssd {

// e^x. kFine (fp32): x log2 e in two parts, since the rounding of the first is 2^-24 of it, some 1e-6 of the
// result far from zero; within 2^-22 of itself. Else that rounding stays: |x| 2^-24 of the result.
template <bool kFine>
__device__ __forceinline__ float exp_of(float x) {
    const float y = x * kLog2e, e = fast_exp2(y);
    if constexpr (!kFine) return e;
    float rest = __builtin_fmaf(x, kLog2e, -y) + x * 1.925963033e-8f;
    rest = fmaxf(rest, -1.f);  // x infinite: not a number until here
    return e * __builtin_fmaf(kLn2, rest, 1.f);
}

// sigmoid(v), and sigmoid(v) with sigmoid(-v), each as exact as the exponential.
template <bool kFine>
__device__ __forceinline__ float sigmoid_of(float v) {
    return __builtin_amdgcn_rcpf(1.f + exp_of<kFine>(-v));
}
struct Gate {
    float s, n;
};
template <bool kFine>
__device__ __forceinline__ Gate gate_of(float v) {
    float e = exp_of<kFine>(-v);
    e = e > 0x1p126f ? 0x1p126f : e;  // sigmoid(v) below 2^-126 counts as 2^-126
    const float s = __builtin_amdgcn_rcpf(1.f + e);
    return {s, e * s};
}

// 1 - e^(2 x) for x <= 0, given e^x: near zero by its series, where the difference would cancel (8 terms to
// x = -1/4: 2^-26 of it; 6 to -1/8: 2^-24).
template <bool kFine>
__device__ __forceinline__ float one_minus_square(float x, float e) {
    const float z = x + x;
    float q;
    if constexpr (kFine) q = 1 / 720.f + z * (1 / 5040.f + z * (1 / 40320.f));
    else q = 1 / 720.f;
    q = 1.f + z * (1 / 2.f + z * (1 / 6.f + z * (1 / 24.f + z * (1 / 120.f + z * q))));
    return z > (kFine ? -0.5f : -0.25f) ? -z * q : __builtin_fmaf(-e, e, 1.f);
}

// A token's decay and its input's coefficient; for the gradients slope = d c / d log a,
// p = d log a / d f and s = sigmoid(f).
struct Decay {
    float a, c, slope, p, s;
};
template <int DECAY, bool kFine, bool kSlopes>
__device__ __forceinline__ Decay decay_of(float f, float rate) {
    Decay o = {};
    if constexpr (DECAY == SSD_DECAY_LOG) {
        o.a = exp_of<kFine>(f);
        o.c = 1.f; o.p = 1.f;
    } else if constexpr (DECAY == SSD_DECAY_SIGMOID) {
        const Gate g = gate_of<kFine>(f);
        o.a = g.s; o.c = g.n; o.slope = -g.s; o.p = g.n;
    } else {
        Gate g = {};
        if constexpr (kSlopes) g = gate_of<kFine>(f);
        else g.s = sigmoid_of<kFine>(f);
        const float la = rate * g.s;
        o.a = exp_of<kFine>(la);
        const float c2 = one_minus_square<kFine>(la, o.a);
        // a decay of 1 (and above: a positive rate) takes no input, and has no slope
        const float r = c2 < 0x1p-100f ? 0.f : __builtin_amdgcn_rsqf(c2);
        o.c = c2 * r; o.slope = -o.a * o.a * r; o.p = la * g.n; o.s = g.s;
    }
    return o;
}

// ---------------------------------------------------------------------------
// A work-group takes a chunk of SSD_GATED_CHUNK tokens of 64 channels. V consecutive channels (16
// bytes) go to a lane, LPR lanes to a token, and R consecutive tokens to each of a wavefront's GPW
// groups of lanes. Where a row ends inside a lane's V channels, that lane takes the row's last V instead: some
// channels then are computed twice, to the same bits. (V = 1: rows of fewer than V.) Loads and stores are of 16
// bytes at any alignment of the type.
// ---------------------------------------------------------------------------
constexpr int kCols = 64, kGatedWaves = 8, kGatedThreads = 64 * kGatedWaves;
template <typename T, int V_>
struct Shape {
    static constexpr int V = V_, LPR = kCols / V, GPW = 64 / LPR, G = GPW * kGatedWaves, R = SSD_GATED_CHUNK / G;
};

template <typename T, int V>
struct Packed {
    typedef uint32_t word __attribute__((ext_vector_type(V * sizeof(T) / 4), aligned(sizeof(T))));
    word w;
    __device__ __forceinline__ void load(const T *p) { w = *reinterpret_cast<const word *>(p); }
    __device__ __forceinline__ float get(int e) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
        return __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
    }
    // Hides from the compiler that the values are those loaded: it would keep what was made of them in registers
    // that it does not have, where making it again is meant.
    __device__ __forceinline__ void forget() {
#pragma unroll
        for (int k = 0; k < V * (int)sizeof(T) / 4; ++k) {
            uint32_t u = w[k];
            asm volatile("" : "+v"(u));
            w[k] = u;
        }
    }
    static __device__ __forceinline__ void store(T *p, const float (&v)[V]) {
        word o;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = __float_as_uint(v[e]);
        } else {
#pragma unroll
            for (int e = 0; e < V / 2; ++e) o[e] = __builtin_bit_cast(uint32_t, bf16x2{(bf16)v[2 * e], (bf16)v[2 * e + 1]});
        }
        *reinterpret_cast<word *>(p) = o;
    }
};
template <typename T>
struct Packed<T, 1> {
    T w;
    __device__ __forceinline__ void load(const T *p) { w = *p; }
    __device__ __forceinline__ float get(int) const { return (float)w; }
    __device__ __forceinline__ void forget() {
        if constexpr (sizeof(T) == 4) {
            asm volatile("" : "+v"(w));
        } else {
            uint32_t u = __builtin_bit_cast(uint16_t, w);
            asm volatile("" : "+v"(u));
            w = __builtin_bit_cast(T, (uint16_t)u);
        }
    }
    static __device__ __forceinline__ void store(T *p, const float (&v)[1]) { *p = (T)v[0]; }
};

// v where keep is all ones, 0 where it is 0, whatever v.
__device__ __forceinline__ float masked(float v, uint32_t keep) { return __uint_as_float(__float_as_uint(v) & keep); }
// A state passed through a piece: decay a (exactly 0 where a reset lies in it), own state h.
__device__ __forceinline__ float pass(float a, float h, float in) { return a == 0.f ? h : __builtin_fmaf(a, in, h); }

// ---------------------------------------------------------------------------
// Handing states on. Work-groups take their chunks by ticket, those of all sequences and columns before the
// next ones along the sequence, so a chunk's predecessors have begun whenever it has. Each publishes its chunk's
// (a, h), waits for the state kWindow chunks back, and passes it through the (a, h) of
// those between, always in this order: the same inputs give the same bits. A word is published once, by one
// store that nothing else has to be ordered with, into memory that k_gated_clear has filled with ones,
// which no published word is.
// ---------------------------------------------------------------------------
constexpr int kWindow = 8;

struct Tile {
    int64_t b;
    int chunk, col;  // along the order of the walk; first channel / kCols
};
// The ticket's chunk (no ticket: a single chunk, which waits for none). Every thread of the work-group calls it.
__device__ __forceinline__ Tile take_tile(uint32_t *ticket, int64_t batch, int cols) {
    __shared__ uint32_t mine;
    uint32_t t = blockIdx.x;
    if (ticket) {
        if (threadIdx.x == 0) mine = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        t = __builtin_amdgcn_readfirstlane(mine);
    }
    const uint32_t wide = (uint32_t)batch * (uint32_t)cols;
    const uint32_t chunk = t / wide, in = t - chunk * wide;
    const uint32_t b = in / (uint32_t)cols;
    return {b, (int)chunk, (int)(in - b * (uint32_t)cols)};
}

__device__ __forceinline__ void publish(uint32_t *word, float v) {
    uint32_t u = __float_as_uint(v);
    u = u == ~0u ? 0x7fc00000u : u;
    __hip_atomic_store(word, u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish(uint64_t *word, float a, float h) {
    uint32_t u = __float_as_uint(h);
    u = u == ~0u ? 0x7fc00000u : u;
    __hip_atomic_store(word, (uint64_t)u << 32 | __float_as_uint(a), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename W>
__device__ __forceinline__ W peek(const W *word) {
    return __hip_atomic_load(word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state that enters chunk k of this lane's column, first being the one that enters chunk 0. pieces and
// ends: the column's words of chunk 0, `stride` apart.
__device__ __forceinline__ float entering(const uint64_t *pieces, const uint32_t *ends, int64_t stride, int k, float first) {
    const int from = k > kWindow ? k - kWindow : 0;
    float h = first;
    if (from > 0) {
        uint32_t u;
        while ((u = peek(ends + (from - 1) * stride)) == ~0u) __builtin_amdgcn_s_sleep(2);
        h = __uint_as_float(u);
    }
    uint64_t w[kWindow];
    for (;;) {
        bool all = true;
#pragma unroll
        for (int j = 0; j < kWindow; ++j) {
            w[j] = 0;
            if (from + j < k) w[j] = peek(pieces + (from + j) * stride);
            all = all && w[j] != ~(uint64_t)0;
        }
        if (all) break;
        __builtin_amdgcn_s_sleep(2);
    }
#pragma unroll
    for (int j = 0; j < kWindow; ++j)
        if (from + j < k) h = pass(__uint_as_float((uint32_t)w[j]), __uint_as_float((uint32_t)(w[j] >> 32)), h);
    return h;
}

// fn(types...) for the call's storage type, decay and whether the input is gated.
template <typename F>
static ssd_status pick_gated(ssd_dtype dtype, int decay, bool in, F fn) {
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
inline ssd_status status_of(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

// Lays the chunks' words out at `workspace`, and has them cleared where there are several chunks (ssd_gated.hip).
ssd_status clear_words(GatedArgs &a, const GatedPlan &p, void *workspace, hipStream_t s);

}  // namespace ssd
