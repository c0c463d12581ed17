// The gated linear recurrence's decay and gates, and how its chunks hand their states on
// (ssd_gated.hip, ssd_gated_bwd.hip).
#pragma once

#include <type_traits>

#include "ssd_common.h"
#include "ssd_internal.h"

namespace ssd {

// v where keep is all ones, 0 where it is 0, whatever v.
__device__ __forceinline__ float masked(float v, uint32_t keep) { return __uint_as_float(__float_as_uint(v) & keep); }

// e^x. kFine (fp32): x log2 e in two parts, since the rounding of the first is 2^-24 of it, some 1e-6 of the
// result far from zero; within 2^-22 of itself. Else that rounding stays: |x| 2^-24 of the result.
template <bool kFine>
__device__ __forceinline__ float exp_of(float x) {
    const float y = x * kLog2e, e = fast_exp2(y);
    if constexpr (!kFine) return e;
    float rest = __builtin_fmaf(x, kLog2e, -y) + x * 1.925963033e-8f;
    rest = fminf(fmaxf(rest, -1.f), 1.f);  // e is 0 or infinite where it is larger, or (x infinite) not a number
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

// 1 - 4^y for y <= 0, given e = 2^y: near zero by its series, where the difference would cancel (8 terms to
// 2 y ln 2 = -1/2: 2^-26 of it; 6 to -1/4: 2^-24).
template <bool kFine>
__device__ __forceinline__ float one_minus_square(float y, float e) {
    constexpr double l = 2 * 0.69314718055994531;
    constexpr float k1 = l, k2 = l * l / 2, k3 = l * l * l / 6, k4 = l * l * l * l / 24, k5 = k4 * l / 5, k6 = k5 * l / 6, k7 = k6 * l / 7,
                    k8 = k7 * l / 8;
    float q = kFine ? k6 + y * (k7 + y * k8) : k6;
    q = k1 + y * (k2 + y * (k3 + y * (k4 + y * (k5 + y * q))));
    return y > (kFine ? -0.36f : -0.18f) ? -y * q : __builtin_fmaf(-e, e, 1.f);
}

// What a token's gate makes: its decay and its input's coefficient. rate2: rate log2 e, at most 0.
struct Decay {
    float a, c;
};
// At a reset (keep 0) nothing passes the decay, whatever the gate. (Of sigmoids and rates c goes by the gate too, and the
// token is undefined where that is.)
template <int DECAY, bool RESET>
__device__ __forceinline__ Decay passed(Decay q, uint32_t keep) {
    return {RESET && DECAY == SSD_DECAY_LOG ? masked(q.a, keep) : q.a, q.c};
}
template <int DECAY, bool kFine>
__device__ __forceinline__ Decay decay_of(float f, float rate2) {
    if constexpr (DECAY == SSD_DECAY_LOG) return {exp_of<kFine>(f), 1.f};
    if constexpr (DECAY == SSD_DECAY_SIGMOID) {
        const Gate g = gate_of<kFine>(f);
        return {g.s, g.n};
    }
    const float y = rate2 * sigmoid_of<kFine>(f), a = fast_exp2(y);
    const float c2 = one_minus_square<kFine>(y, a);
    return {a, c2 * __builtin_amdgcn_rsqf(c2 + 0x1p-126f)};  // 0 where c2 is
}
// A positive rate counts as 0; in two steps, so that its rounding does not follow that of the product.
__device__ __forceinline__ float base2(float rate) { return (rate > 0.f ? 0.f : rate) * kLog2e; }

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
    // Set in ascending order, two to a word in 16 bits. Formed here and now: the compiler would put the last steps
    // off to the store, and keep what they are made of until then.
    __device__ __forceinline__ void set(int e, float v) {
        if (sizeof(T) == 2 && !(e & 1)) {
            w[e >> 1] = __float_as_uint(v);
            return;
        }
        uint32_t u = __float_as_uint(v);
        if constexpr (sizeof(T) == 2) u = __builtin_bit_cast(uint32_t, bf16x2{(bf16)__uint_as_float(w[e >> 1]), (bf16)v});
        asm volatile("" : "+v"(u));
        w[e * (int)sizeof(T) / 4] = u;
    }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<word *>(p) = w; }
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
    __device__ __forceinline__ void set(int, float v) {
        w = (T)v;
        forget();
    }
    __device__ __forceinline__ void store(T *p) const { *p = w; }
};

// A tensor's tokens from a chunk's first one on: token i's channel d at a 32-bit offset from one address
// for the work-group.
template <typename T>
struct Tokens {
    const char *p;
    uint32_t ld, at;  // bytes
    __device__ __forceinline__ Tokens(const void *q, int64_t row, int64_t ld_, int i, int d)
        : p(reinterpret_cast<const char *>(q) + row * ld_ * (int64_t)sizeof(T)), ld((uint32_t)ld_ * (uint32_t)sizeof(T)) {
        asm volatile("" : "+v"(i));  // made for every tile: kept over them, the tensors' offsets would not fit the registers
        at = (uint32_t)i * ld + (uint32_t)d * (uint32_t)sizeof(T);
    }
    __device__ __forceinline__ const T *operator[](int r) const { return reinterpret_cast<const T *>(p + (uint32_t)r * ld + at); }
    __device__ __forceinline__ T *out(int r) const { return const_cast<T *>((*this)[r]); }
};

// A piece's decay where a reset lies in it: -0, which no product of decays is. It stays that whatever the piece's other
// decays are: a plain product with one that is undefined or infinite would not be zero, and would let in what a reset leaves out.
constexpr uint32_t kMark = 0x80000000u;
__device__ __forceinline__ bool marked(float a) { return __float_as_uint(a) == kMark; }
// a where open is all ones, the mark where it is 0; and the decay of two pieces, one after the other
template <bool RESET>
__device__ __forceinline__ float mark(float a, uint32_t open) {
    return RESET ? __uint_as_float((__float_as_uint(a) & open) | (kMark & ~open)) : a;
}
template <bool RESET>
__device__ __forceinline__ float join(float a, float b) {
    return RESET && (marked(a) || marked(b)) ? __uint_as_float(kMark) : a * b;
}
// A state passed through a piece: decay a, own state h. Where a is the mark, what enters may be anything; decays
// that underflow are no reset, and an undefined state goes on through them.
template <bool RESET>
__device__ __forceinline__ float pass(float a, float h, float in) {
    return RESET && marked(a) ? h : __builtin_fmaf(a, in, h);
}
template <bool RESET>
__device__ __forceinline__ float cut(float v, uint32_t keep) { return RESET ? masked(v, keep) : v; }

// ---------------------------------------------------------------------------
// Handing states on. Work-groups take their chunks by ticket, those of all sequences and columns before the
// next ones along the sequence, so a chunk's predecessors belong to work-groups that have begun whenever it does, and
// that wait for earlier chunks only: every wait ends. Tickets are given out one each 13 ns, as long as a small tile takes the
// memory; where tiles are so small a ticket is for two of a chunk, one after the other. Each publishes its chunk's
// (a, h), waits for the state kWindow chunks back, and passes it through the (a, h) of
// those between, always in this order: the same inputs give the same bits. A word is published once, by one
// store that nothing else has to be ordered with, into memory that k_gated_clear has filled with ones,
// which no published word is.
// ---------------------------------------------------------------------------
constexpr int kWindow = 3;
// Looks that a wait gives up after, some seconds: it ends by the order of the tickets, unless the words are overwritten
// while the kernel runs (a workspace that another call uses at the same time). Results are NaN then.
constexpr int kMostLooks = 1 << 22;

struct Tile {
    int64_t b;
    int chunk, col;  // along the order of the walk; first channel / kCols
};
// A kernel's arguments where the launch put them, its only ones. They are read where they are needed, again() and
// again: over the tiles' loop they are more than the scalar registers hold, and a hundred of a tile's vector instructions
// moved them to lanes and back.
typedef const __attribute__((address_space(4))) GatedArgs *Args;
__device__ __forceinline__ Args args() { return (Args)__builtin_amdgcn_kernarg_segment_ptr(); }
__device__ __forceinline__ void again(Args &a) { asm volatile("" : "+s"(a)); }

// A work-group's way through its tiles, `share` to a ticket, of one chunk (no ticket: one tile, of a single chunk, which
// waits for none). Every thread holds the same.
struct Way {
    uint32_t chunk, now, end;  // of the chunk's tiles of all sequences and columns: this one, and the ticket's end
    __device__ __forceinline__ Way(Args a, uint32_t *mine) {
        uint32_t t = blockIdx.x;
        if (a->ticket) {
            if (threadIdx.x == 0) *mine = __hip_atomic_fetch_add(a->ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __syncthreads();
            t = __builtin_amdgcn_readfirstlane(*mine);
            __syncthreads();
        }
        set(a, t);
    }
    __device__ __forceinline__ void set(Args a, uint32_t t) {
        chunk = t / a->tickets;
        now = (t - chunk * a->tickets) * a->share;
        end = min(now + a->share, a->wide);
    }
    __device__ __forceinline__ Tile tile(uint32_t cols) const {
        const uint32_t b = now / cols;
        return {b, (int)chunk, (int)(now - b * cols)};
    }
    // The next ticket, where the last tile of one is under way: ask() for it early (thread 0 holds the answer),
    // tell() it to the others in front of a barrier, go_on() behind that.
    __device__ __forceinline__ uint32_t ask(Args a) const {
        if (a->ticket && now + 1 >= end && threadIdx.x == 0)
            return __hip_atomic_fetch_add(a->ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        return 0;
    }
    __device__ __forceinline__ void tell(uint32_t next, uint32_t *mine) const {
        if (now + 1 >= end && threadIdx.x == 0) *mine = next;
    }
    __device__ __forceinline__ void go_on(Args a, const uint32_t *mine) {
        if (++now < end) return;
        if (a->ticket) set(a, __builtin_amdgcn_readfirstlane(*mine));
        else chunk = (uint32_t)a->nchunks;
    }
};

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

// The words from which the state that enters chunk k of this lane's column follows: the state kWindow chunks back (none
// where the sequence begins within them), and the pieces since. pieces and ends: the columns' words of chunk 0,
// `stride` apart. look() asks for them, and state() waits, looking again where one was not there yet; loads that the
// wavefront issues in between, and whose results are further away, do not stand in the way of the first look.
template <bool RESET>
struct Entering {
    uint64_t w[kWindow];
    uint32_t end;
    __device__ __forceinline__ void look(const uint64_t *pieces, const uint32_t *ends, int64_t stride, int lane, int k) {
        const int from = max(k - kWindow, 0);
        asm volatile("" : "+v"(lane));  // the addresses are made here: in front of the tiles' loop they took registers all the way
        end = 0;
        if (from > 0) end = peek(ends + (from - 1) * stride + lane);
#pragma unroll
        for (int j = 0; j < kWindow; ++j) {
            w[j] = 0;
            if (from + j < k) w[j] = peek(pieces + (from + j) * stride + lane);
        }
    }
    // first: what enters chunk 0
    __device__ __forceinline__ float state(const uint64_t *pieces, const uint32_t *ends, int64_t stride, int lane, int k, float first) {
        for (int looks = 0;; ++looks) {
            bool all = end != ~0u;
#pragma unroll
            for (int j = 0; j < kWindow; ++j) all = all && w[j] != ~(uint64_t)0;
            if (all) break;
            if (looks == kMostLooks) return __builtin_nanf("");
            __builtin_amdgcn_s_sleep(1);
            look(pieces, ends, stride, lane, k);
        }
        float h = k > kWindow ? __uint_as_float(end) : first;
#pragma unroll
        for (int j = 0; j < kWindow; ++j)
            if (max(k - kWindow, 0) + j < k) h = pass<RESET>(__uint_as_float((uint32_t)w[j]), __uint_as_float((uint32_t)(w[j] >> 32)), h);
        return h;
    }
};

// fn(types...) for the call's storage type, decay, whether the input is gated and whether there are resets.
template <typename F>
static ssd_status pick_gated(ssd_dtype dtype, int decay, bool in, bool reset, F fn) {
    auto two = [&](auto t, auto dec) {
        if (reset) return in ? fn(t, dec, std::true_type{}, std::true_type{}) : fn(t, dec, std::false_type{}, std::true_type{});
        return in ? fn(t, dec, std::true_type{}, std::false_type{}) : fn(t, dec, std::false_type{}, std::false_type{});
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
