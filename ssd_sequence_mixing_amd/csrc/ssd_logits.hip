// What a decoder does to its logits before it chooses, for gfx950. With n(v) how
// often token v stands in a row's history, and g(v) how often behind its prompt:
//
//   l(v) <- l > 0 ? l / repetition : l * repetition      where n(v) > 0
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

template <typename T, int SLICE, bool HISTORY, bool DENSE>
__global__ __launch_bounds__(kLogitThreads) void k_logits(LogitsArgs a) {
    constexpr int E = 16 / (int)sizeof(T);
    typedef float f32_any __attribute__((aligned(4)));
    __shared__ __attribute__((aligned(16))) uint32_t count[HISTORY ? SLICE : 4];
    const int64_t row = blockIdx.x / a.slices;
    const int64_t V = a.vocab, at = row * V;
    // slices begin where a row has 16 aligned bytes: the first one is shorter by what lies before that
    const int lead = (int)(at & (E - 1));
    const int64_t v0 = (int64_t)(blockIdx.x - row * a.slices) * SLICE - lead;  // the slice's place 0
    float rep = 1.f, pres = 0.f, freq = 0.f;
    if constexpr (HISTORY) {
        for (int i = threadIdx.x * 4; i < SLICE; i += kLogitThreads * 4) *reinterpret_cast<u32x4 *>(count + i) = u32x4{0, 0, 0, 0};
        if (a.repetition) rep = a.repetition[row];
        if (a.presence) pres = a.presence[row];
        if (a.frequency) freq = a.frequency[row];
        const int64_t cap = a.capacity;
        int64_t len = a.lengths ? a.lengths[row] : cap, prompt = a.prompt ? a.prompt[row] : 0;
        len = len < 0 ? 0 : len > cap ? cap : len;
        const int *h = a.tokens + row * cap;
        __syncthreads();
        for (int64_t i = threadIdx.x; i < len; i += kLogitThreads) {
            const int64_t t = (int64_t)h[i] - v0;
            if (t >= 0 && t < SLICE && (uint32_t)h[i] < (uint32_t)V) {
                atomicOr(&count[t], kSeen);
                if (i >= prompt) atomicAdd(&count[t], 1u);
            }
        }
        __syncthreads();
    }
    const T *in = reinterpret_cast<const T *>(a.logits) + at;
    T *out = reinterpret_cast<T *>(a.out) + at;
    const float *bias = DENSE && a.bias ? a.bias + (a.bias_rows > 1 ? at : 0) : nullptr;
    const uint32_t *mask = DENSE && a.mask ? a.mask + (a.mask_rows > 1 ? row * a.words : 0) : nullptr;
    auto value = [&](float l, int64_t v, uint32_t c, bool &touched) {
        touched = false;
        if (HISTORY && c) {
            const uint32_t n = c & (kSeen - 1);
            l = l > 0.f ? l / rep : l * rep;
            if (n) l -= freq * (float)n + pres;
            touched = true;
        }
        if constexpr (DENSE) {
            if (bias) l += bias[v], touched = true;
            if (mask && !(mask[v >> 5] >> (v & 31) & 1)) l = -INFINITY, touched = true;
        }
        return l;
    };
    for (int i = threadIdx.x * E; i < SLICE; i += kLogitThreads * E) {
        const int64_t v = v0 + i;
        if (v >= V) break;
        union {
            T e[E];
            u32x4 q;
        } x;
        const bool whole = v >= 0 && v + E <= V;
        if (whole) {
            x.q = *reinterpret_cast<const u32x4 *>(in + v);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) x.e[e] = v + e >= 0 && v + e < V ? in[v + e] : (T)0.f;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (!whole && (v + e < 0 || v + e >= V)) continue;
            bool touched;
            const float l = value((float)x.e[e], v + e, HISTORY ? count[i + e] : 0u, touched);
            if (touched) x.e[e] = (T)l;  // others keep their bits
        }
        if (whole) {
            *reinterpret_cast<u32x4 *>(out + v) = x.q;
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (v + e >= 0 && v + e < V) out[v + e] = x.e[e];
        }
    }
}

constexpr int kSlice = 4096;
int64_t logits_slices(int64_t vocab) { return (vocab + 7 + kSlice - 1) / kSlice; }  // with up to 7 places before the first

ssd_status launch_logits(LogitsArgs a, ssd_dtype dtype, hipStream_t s) {
    a.slices = (int)logits_slices(a.vocab);
    auto go = [&](auto t, auto h, auto d) {
        return launch(k_logits<decltype(t), kSlice, decltype(h)::value, decltype(d)::value>, dim3((unsigned)(a.rows * a.slices)),
                      dim3(kLogitThreads), s, a) == hipSuccess
                   ? SSD_OK
                   : SSD_ERR_HIP;
    };
    auto by = [&](auto t) {
        const bool dense = a.bias || a.mask;
        if (a.tokens) return dense ? go(t, std::true_type{}, std::true_type{}) : go(t, std::true_type{}, std::false_type{});
        return dense ? go(t, std::false_type{}, std::true_type{}) : go(t, std::false_type{}, std::false_type{});
    };
    return dtype == SSD_BF16 ? by(bf16{}) : by(float{});
}

}  // namespace ssd
