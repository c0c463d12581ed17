// What a decoder does to its logits before it chooses, for gfx950. With n(v) how
// often token v stands in a row's history, and g(v) how often behind its prompt:
//
//   l(v) <- l > 0 ? l / repetition : l * repetition      where n(v) > 0 (by the inverse, where that is an ordinary number)
//   l(v) <- l - frequency g(v) - presence                where g(v) > 0
//   l(v) <- l + bias(v);   -inf where the mask's bit v is 0
//
// A work-group takes a slice of a row's vocabulary. It counts the history's tokens
// that lie in it in LDS (integer atomics: no order matters), then passes over the slice once,
// 16 bytes a lane. Bound: HBM, one read and one write of the logits.
#include <type_traits>

#include "ssd_common.h"
#include "ssd_internal.h"

namespace ssd {

constexpr int kLogitThreads = 256;
constexpr uint32_t kSeen = 1u << 31;  // beside the count behind the prompt: the token stands in the history

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(4)));

// HISTORY: there are tokens; DENSE: there is a bias or a mask.
template <typename T, int SLICE, bool HISTORY, bool DENSE>
__global__ __launch_bounds__(kLogitThreads) void k_logits(LogitsArgs a) {
    constexpr int E = 16 / (int)sizeof(T);
    __shared__ __attribute__((aligned(16))) uint32_t count[HISTORY ? SLICE : 4];
    const int64_t row = blockIdx.x / a.slices, V = a.vocab, at = row * V;
    // slices begin where a row has 16 aligned bytes: the first one is shorter by what lies before that
    const int lead = (int)(at & (E - 1));
    const int64_t v0 = (int64_t)(blockIdx.x - row * a.slices) * SLICE - lead;  // the slice's place 0
    const T *in = reinterpret_cast<const T *>(a.logits) + at;
    T *out = reinterpret_cast<T *>(a.out) + at;
    union Group {
        T e[E];
        u32x4 q;
    };
    // every whole group of the slice is on its way before the history is looked at (loads and stores past the caches,
    // which 64 x 8 x 65536 logits do not fit: 80 us without, 65 so)
    constexpr int N = SLICE / (kLogitThreads * E);
    const int64_t left = V - v0;
    const int whole_from = v0 < 0 ? E : 0, whole_to = (int)(left < SLICE ? left / E * E : SLICE);
    auto place = [&](int k) { return (k * kLogitThreads + (int)threadIdx.x) * E; };
    auto whole = [&](int p) { return p >= whole_from && p + E <= whole_to; };
    Group x[N];
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (whole(place(k))) x[k].q = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(in + v0 + place(k)));
    float rep = 1.f, inv = 1.f, pres = 0.f, freq = 0.f;
    bool plain = true;  // the inverse is an ordinary number
    if constexpr (HISTORY) {
        for (int i = threadIdx.x * 4; i < SLICE; i += kLogitThreads * 4) *reinterpret_cast<u32x4 *>(count + i) = u32x4{0, 0, 0, 0};
        if (a.repetition) rep = a.repetition[row], inv = 1.f / rep, plain = rep >= 0x1p-126f && rep <= 0x1p126f;
        if (a.presence) pres = a.presence[row];
        if (a.frequency) freq = a.frequency[row];
        const int cap = (int)a.capacity;
        int len = a.lengths ? a.lengths[row] : cap;
        const int prompt = a.prompt ? a.prompt[row] : 0;
        len = len < 0 ? 0 : len > cap ? cap : len;
        const int *h = a.tokens + row * cap;
        const int64_t end = min(V, v0 + SLICE);
        __syncthreads();
        auto seen = [&](int token, int64_t i) {
            if (token >= 0 && token >= v0 && token < end) {
                uint32_t *c = &count[token - v0];
                atomicOr(c, kSeen);
                if (i >= prompt) atomicAdd(c, 1u);
            }
        };
        int64_t i = threadIdx.x * 4;
        for (; i + 4 <= len; i += kLogitThreads * 4) {
            const u32x4_any t = *reinterpret_cast<const u32x4_any *>(h + i);
#pragma unroll
            for (int k = 0; k < 4; ++k) seen((int)t[k], i + k);
        }
        for (int64_t k = i; k < len && k < i + 4; ++k) seen(h[k], k);
        __syncthreads();
    }
    const float *bias = DENSE && a.bias ? a.bias + (a.bias_rows > 1 ? at : 0) : nullptr;
    const uint32_t *mask = DENSE && a.mask ? a.mask + (a.mask_rows > 1 ? row * a.words : 0) : nullptr;
    // what becomes of the logits of places i .. i + E - 1 of the slice, tokens v and on; others keep their bits
    auto apply = [&](Group &x, int i, int64_t v, auto all, auto by_inverse) {
        constexpr bool kAll = decltype(all)::value, kInverse = decltype(by_inverse)::value;
        float l[E];
#pragma unroll
        for (int e = 0; e < E; ++e) l[e] = (float)x.e[e];
        bool touched[E] = {};
        if constexpr (HISTORY) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const uint32_t c = count[i + e], n = c & (kSeen - 1);
                const float less = n ? __builtin_fmaf(freq, (float)n, pres) : 0.f;
                const float scaled = kInverse ? l[e] * (l[e] > 0.f ? inv : rep) : l[e] > 0.f ? l[e] / rep : l[e] * rep;
                l[e] = c ? scaled - less : l[e];
                touched[e] = c != 0;
            }
        }
        if constexpr (DENSE) {
            if (bias) {
                if constexpr (kAll) {
#pragma unroll
                    for (int k = 0; k < E; k += 4) {
                        const u32x4_any b = *reinterpret_cast<const u32x4_any *>(bias + v + k);
#pragma unroll
                        for (int e = 0; e < 4; ++e) l[k + e] += __uint_as_float(b[e]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (v + e >= 0 && v + e < V) l[e] += bias[v + e];
                }
#pragma unroll
                for (int e = 0; e < E; ++e) touched[e] = true;
            }
            if (mask) {
                // the two words that the E bits lie in
                const int64_t first = v < 0 ? 0 : v >> 5, last = a.words - 1;
                const uint64_t both = (uint64_t)mask[min(first + 1, last)] << 32 | mask[min(first, last)];
                const uint32_t bits = v < 0 ? (uint32_t)both << (uint32_t)-v : (uint32_t)(both >> (v & 31));
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const bool shut = !(bits >> e & 1);
                    l[e] = shut ? -INFINITY : l[e];
                    touched[e] |= shut;
                }
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) x.e[e] = touched[e] ? (T)l[e] : x.e[e];
    };
    auto wholes = [&](auto by_inverse) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int p = place(k);
            if (whole(p)) {
                apply(x[k], p, v0 + p, std::true_type{}, by_inverse);
                __builtin_nontemporal_store(x[k].q, reinterpret_cast<u32x4 *>(out + v0 + p));
            }
        }
    };
    // a division of every logit took 52 us where this takes 49 (512 x 65536 in fp32), and a branch at each 51
    if (plain) wholes(std::true_type{});
    else wholes(std::false_type{});
    // a group that the row begins or ends in
    const int tail = left > 0 && left < SLICE && whole_to >= whole_from && left % E ? whole_to : -1;
    const int mine = threadIdx.x == 0 && whole_from ? 0 : threadIdx.x == 1 && tail >= 0 ? tail : -1;
    if (mine >= 0) {
        const int64_t v = v0 + mine;
        Group y;
#pragma unroll
        for (int e = 0; e < E; ++e) y.e[e] = v + e >= 0 && v + e < V ? in[v + e] : (T)0.f;
        if (plain) apply(y, mine, v, std::false_type{}, std::true_type{});
        else apply(y, mine, v, std::false_type{}, std::false_type{});
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (v + e >= 0 && v + e < V) out[v + e] = y.e[e];
    }
}

// Slices of 8192 logits, or of 2048 where those would be fewer than two work-groups for each CU.
static int64_t slices_of(int64_t vocab, int64_t slice) { return (vocab + 7 + slice - 1) / slice; }  // with up to 7 places before the first
int64_t logits_slices(int64_t vocab) { return slices_of(vocab, 2048); }

ssd_status launch_logits(LogitsArgs a, ssd_dtype dtype, hipStream_t s) {
    auto go = [&](auto t, auto slice, auto h, auto d) {
        constexpr int SLICE = decltype(slice)::value;
        a.slices = (int)slices_of(a.vocab, SLICE);
        return launch(k_logits<decltype(t), SLICE, decltype(h)::value, decltype(d)::value>, dim3((unsigned)(a.rows * a.slices)),
                      dim3(kLogitThreads), s, a) == hipSuccess
                   ? SSD_OK
                   : SSD_ERR_HIP;
    };
    auto by = [&](auto t, auto slice) {
        const bool dense = a.bias || a.mask;
        if (a.tokens) return dense ? go(t, slice, std::true_type{}, std::true_type{}) : go(t, slice, std::true_type{}, std::false_type{});
        return dense ? go(t, slice, std::false_type{}, std::true_type{}) : go(t, slice, std::false_type{}, std::false_type{});
    };
    auto of = [&](auto t) {
        if (a.rows * slices_of(a.vocab, 8192) >= 512) return by(t, std::integral_constant<int, 8192>{});
        return by(t, std::integral_constant<int, 2048>{});
    };
    return dtype == SSD_BF16 ? of(bf16{}) : of(float{});
}

}  // namespace ssd
