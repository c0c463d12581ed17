// Rows in 8-bit integers for gfx950: scale = max |x| / 127 of the row, and
// q the integer nearest to x / scale (ties to even). A row of zeros has scale 0; one that holds an
// infinity or a NaN has scale NaN, and codes 0.
#include <type_traits>

#include "ssd_common.h"
#include "ssd_internal.h"

namespace ssd {

// The integer nearest to x / s, |x| <= 127 s (1 + 2^-24): the rounded quotient's, put right by
// the remainder x - q s, which is exact in one fused operation (a multiple of the smaller operand's last place below s).
__device__ __forceinline__ int code_of(float x, float s) {
    float q = rintf(x / s);
    const float r = __builtin_fmaf(-q, s, x), half = 0.5f * s;
    const bool odd = ((int)q & 1) != 0;
    if (r > half || (r == half && odd)) q += 1.f;
    else if (r < -half || (r == -half && odd)) q -= 1.f;
    return (int)fminf(fmaxf(q, -127.f), 127.f);
}

template <typename T>
__global__ __launch_bounds__(256) void k_int_quantize(const T *x, int8_t *q, float *scale, int64_t rows, int dim) {
    __shared__ float tops[4];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T *p = x + r * dim;
        float top = 0.f;
        bool bad = false;
        for (int d = threadIdx.x; d < dim; d += 256) {
            const float v = fabsf((float)p[d]);
            bad |= !(v < INFINITY);
            top = fmaxf(top, v);
        }
        top = bad ? INFINITY : top;
        for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
        __syncthreads();
        if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
        __syncthreads();
        top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        bad = top == INFINITY;
        const float s = top / 127.f;
        for (int d = threadIdx.x; d < dim; d += 256) q[r * dim + d] = bad || s == 0.f ? 0 : (int8_t)code_of((float)p[d], s);
        if (threadIdx.x == 0) scale[r] = bad ? __builtin_nanf("") : s;
    }
}

ssd_status launch_int_quantize(const void *x, int8_t *q, float *scale, int64_t rows, int64_t dim, ssd_dtype dtype, hipStream_t s) {
    auto go = [&](auto t) {
        using T = decltype(t);
        const int64_t most = 1 << 20;
        return launch(k_int_quantize<T>, dim3((unsigned)(rows < most ? rows : most)), dim3(256), s, (const T *)x, q, scale, rows, (int)dim) ==
                       hipSuccess
                   ? SSD_OK
                   : SSD_ERR_HIP;
    };
    return dtype == SSD_BF16 ? go(bf16{}) : go(float{});
}

}  // namespace ssd
