// Rows in 8-bit integers for gfx950: scale = max |x| / 127 of the row (times the fp32 number nearest to 1 / 127), and
// q the integer nearest to x / scale (ties to even). A row of zeros has scale 0; one that holds an
// infinity or a NaN has scale NaN, and codes 0.
//
// A row stays in the registers of one wavefront (many rows) or of 4 or 16, 8 values a lane and load, at any
// alignment; rows of more than 65536 values are read twice. Bound: HBM, one read and one write.
// A code is formed by the scale's inverse, and is at most 1 off; the exact remainder, half a scale or more, says where.
// (With the maximum in fp32 and every value of a wavefront's decided again where one lay in the middle, 30 operations a
// value, the vector unit was busy 94% of the time.)
#include <type_traits>

#include "ssd_common.h"
#include "ssd_internal.h"

namespace ssd {

// The integer nearest to x / s, ties to even: one that is at most 1 off, put right by the remainder x - q s, which one
// fused operation gives exactly (a multiple of the smaller operand's last place, and below 2 s).
__device__ __forceinline__ float nearest(float x, float s) {
    float q = rintf(x / s);
    const float r = 2.f * __builtin_fmaf(-q, s, x);  // (half of a scale of few bits would be rounded)
    const bool odd = ((int)q & 1) != 0;
    if (r > s || (r == s && odd)) q += 1.f;
    else if (r < -s || (r == -s && odd)) q -= 1.f;
    return q;
}

// 8 values of a row, as stored.
template <typename T>
struct Eight {
    static constexpr int kWords = 2 * (int)sizeof(T);
    uint32_t w[kWords];
    __device__ __forceinline__ float get(int e) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
        return __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
    }
    // Hides from the compiler that the values are those loaded: it would keep them unpacked, in twice the registers.
    __device__ __forceinline__ void forget() {
#pragma unroll
        for (int k = 0; k < kWords; ++k) asm volatile("" : "+v"(w[k]));
    }
    // values from p on, zeros from n on
    __device__ __forceinline__ void load(const T *p, int n) {
        typedef uint32_t word __attribute__((ext_vector_type(4), aligned(2)));
        if (n >= 8) {
#pragma unroll
            for (int k = 0; k < kWords; k += 4) {
                // past the caches: the product that follows then finds more of the codes there (8192 x 4096, and 4096 x 2048
                // behind it: 116 us without, 106 so, though this alone took 30 and not 27)
                const word q = __builtin_nontemporal_load(reinterpret_cast<const word *>(reinterpret_cast<const char *>(p) + 4 * k));
#pragma unroll
                for (int e = 0; e < 4; ++e) w[k + e] = q[e];
            }
        } else {
            T v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < n ? p[e] : (T)0.f;
            __builtin_memcpy(w, v, sizeof v);
        }
    }
    // The larger of top and their magnitudes' bits (in 16 bits: two by two), in which an infinity or a NaN lies above all others.
    __device__ __forceinline__ void largest(uint32_t &top) const {
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            if constexpr (sizeof(T) == 4) {
                top = max(top, w[k] & 0x7fffffffu);
            } else {
                typedef uint16_t two __attribute__((ext_vector_type(2)));
                top = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(two, top), __builtin_bit_cast(two, w[k] & 0x7fff7fffu)));
            }
        }
    }
    static __device__ __forceinline__ uint32_t as_float(uint32_t top) {
        if constexpr (sizeof(T) == 4) return top;
        return max(top >> 16, top & 0xffffu) << 16;
    }
    // Their codes to q, n of them. inv: 1 / s or next to it, where that is an ordinary number, or 0.
    __device__ __forceinline__ void store(int8_t *q, int n, float s, float inv, bool zero) const {
        constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, which is the sum's lowest byte
        uint32_t u[8];
        if (__any(inv == 0.f)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = __float_as_uint(fminf(fmaxf(nearest(get(e), s), -127.f), 127.f) + kMagic);  // a scale of few bits may be far below its value
        } else {
            const float half = 0.5f * s;
            float rest[8], far = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float r = __builtin_fmaf(get(e), inv, kMagic);
                rest[e] = __builtin_fmaf(-(r - kMagic), s, get(e));
                far = fmaxf(far, fabsf(rest[e]));
                u[e] = __float_as_uint(r);
            }
            // as nearest(); value by value, since they are few (in bf16 half the rows' largest value, which lies in the middle)
            if (__any(far >= half)) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (__any(fabsf(rest[e]) >= half)) {
                        const bool next = fabsf(rest[e]) > half || (fabsf(rest[e]) == half && (u[e] & 1));
                        u[e] += next ? (rest[e] > 0.f ? 1u : ~0u) : 0u;
                    }
            }
        }
        uint32_t o[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t lo = __builtin_amdgcn_perm(u[4 * k + 1], u[4 * k], 0x0c0c0400u);
            const uint32_t hi = __builtin_amdgcn_perm(u[4 * k + 3], u[4 * k + 2], 0x04000c0cu);
            o[k] = zero ? 0u : lo | hi;
        }
        typedef uint32_t pair __attribute__((ext_vector_type(2), aligned(1)));
        if (n >= 8) {
            *reinterpret_cast<pair *>(q) = pair{o[0], o[1]};
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) q[e] = (int8_t)(o[e >> 2] >> (8 * (e & 3)));
        }
    }
};

// W wavefronts a row (at most 4 of them: 4 / W rows a work-group), NC loads a lane. NC = 0: rows read twice.
template <typename T, int W, int NC>
__global__ __launch_bounds__(W > 4 ? 64 * W : 256) void k_int_quantize(const T *x, int8_t *q, float *scale, int64_t rows, int dim) {
    constexpr int RPB = W > 4 ? 1 : 4 / W, kStep = 64 * W * 8;
    __shared__ uint32_t tops[W > 1 ? W : 1];
    const int t = threadIdx.x % (64 * W), slot = threadIdx.x / (64 * W);
    const int64_t hop = (int64_t)gridDim.x * RPB;
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < rows; r0 += hop) {
        const int64_t r = r0 + slot;
        const bool in = r < rows;
        const T *p = x + (in ? r : 0) * dim;
        const int n = in ? dim : 0;
        Eight<T> v[NC ? NC : 1];
        uint32_t top = 0;
        if constexpr (NC > 0) {
#pragma unroll
            for (int c = 0; c < NC; ++c) v[c].load(p + min(c * kStep + t * 8, dim), n - (c * kStep + t * 8));
#pragma unroll
            for (int c = 0; c < NC; ++c) v[c].largest(top);
        } else {
            for (int d = t * 8; d < n; d += kStep) {
                v[0].load(p + d, n - d);
                v[0].largest(top);
            }
        }
        top = Eight<T>::as_float(top);
#pragma unroll
        for (int o = 32; o; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
        if constexpr (W > 1) {
            if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < W; ++k) top = max(top, tops[k]);
            __syncthreads();
        }
        if constexpr (NC > 0) {
#pragma unroll
            for (int c = 0; c < NC; ++c) v[c].forget();
        }
        const bool bad = top >= 0x7f800000u;
        const float s = __uint_as_float(top) * (1.f / 127.f), inv = s > 0x1p-100f && !bad ? __builtin_amdgcn_rcpf(s) : 0.f;
        const bool zero = bad || s == 0.f;
        int8_t *o = q + (in ? r : 0) * dim;
        if constexpr (NC > 0) {
#pragma unroll
            for (int c = 0; c < NC; ++c) v[c].store(o + min(c * kStep + t * 8, dim), n - (c * kStep + t * 8), s, inv, zero);
        } else {
            for (int d = t * 8; d < n; d += kStep) {
                v[0].load(p + d, n - d);
                v[0].store(o + d, n - d, s, inv, zero);
            }
        }
        if (in && t == 0) scale[r] = bad ? __builtin_nanf("") : s;
    }
}

ssd_status launch_int_quantize(const void *x, int8_t *q, float *scale, int64_t rows, int64_t dim, ssd_dtype dtype, hipStream_t s) {
    auto of = [&](auto t) {
        using T = decltype(t);
        auto go = [&](auto k, int W) {
            const int64_t per = W > 4 ? 1 : 4 / W, blocks = (rows + per - 1) / per, most = 1 << 20;
            return launch(k, dim3((unsigned)(blocks < most ? blocks : most)), dim3(W > 4 ? 64 * W : 256), s, (const T *)x, q, scale, rows,
                          (int)dim) == hipSuccess
                       ? SSD_OK
                       : SSD_ERR_HIP;
        };
        // short rows: one wavefront each, if there are rows for every SIMD. Else 4 wavefronts a row, of 1 to 4 loads a
        // lane (8192 x 4096 in bf16: 22 us, 4.6 TB/s; with one wavefront of 8 loads 37 where this took 26), or 16 of them
        const int64_t c = (dim + 511) / 512;
        if (c == 1) return go(k_int_quantize<T, 1, 1>, 1);
        if (c == 2 && rows >= 1024) return go(k_int_quantize<T, 1, 2>, 1);
        if (c <= 4) return go(k_int_quantize<T, 4, 1>, 4);
        if (c <= 8) return go(k_int_quantize<T, 4, 2>, 4);
        if (c <= 16) return go(k_int_quantize<T, 4, 4>, 4);
        if (c <= 32) return go(k_int_quantize<T, 16, 2>, 16);
        if (c <= 64) return go(k_int_quantize<T, 16, 4>, 16);
        if (c <= 128) return go(k_int_quantize<T, 16, 8>, 16);
        return go(k_int_quantize<T, 16, 0>, 16);
    };
    return dtype == SSD_BF16 ? of(bf16{}) : of(float{});
}

}  // namespace ssd
