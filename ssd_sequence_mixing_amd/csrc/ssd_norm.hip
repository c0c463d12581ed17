// Root-mean-square norm of a layer's rows for gfx950, with the residual's
// addition in front and an 8-bit output behind, its backward pass, and the
// 8-bit quantiser by itself.
//
//   h = x + r;  inv = 1 / sqrt(mean(h^2) + eps);  y = h inv w
//
// over each of `groups` equal pieces of a row of D values (a tensor-parallel
// layer's norm takes one piece per group). Everything is held in fp32; r's
// sum is rounded once, to the stored h, and y once, to its storage type.
//
// 8 bits: every 32 consecutive y share a power of two 2^p, p the smallest
// whole number >= -127 with max|y| <= 448 * 2^p (448 is e4m3's largest value,
// so nothing saturates and nothing is clipped), stored as p + 127 (e8m0), and
// the code of y is e4m3(y 2^-p), rounded to nearest even; y 2^-p is exact. These are
// the operands the matrix cores' scaled products take as they are. In between y is
// formed to 48 bits and rounded to odd, and inv's rest is kept, so that a code is the
// nearest one to h inv w and not to its fp32 rounding: of 16.8 million codes (8192 x
// 2048) 2 differ from the formula's in 64 bits, and 12 without that, for 2 us of 37.
// A block that holds a value that is not finite gets the scale 255 (NaN) and codes 0x7f (NaN).
//
// Bound: HBM, one read and one write of every row. A row stays in registers
// between the sum and the scaling, so it is read once: W wavefronts take one
// row, each lane NC chunks of 8 consecutive values (one 16-byte load in bf16).
// With many rows one wavefront takes a row (no barrier, NC loads in flight);
// with few rows the time is latency, and a row is spread over 4.
// 8192 x 2048, fp32 residual, 8-bit output: 189 MB in 36 us, 5.3 TB/s; one row
// of 2048: 2.3 us.
#include <type_traits>

#include "ssd_common.h"
#include "ssd_internal.h"

namespace ssd {

constexpr int kNormThreads = 256;

// 8 values of one chunk as fp32. V: the chunk is 8 consecutive values, 16-byte
// aligned; else the values are taken one by one, `step` apart, where i < n.
template <typename T, bool V>
__device__ __forceinline__ void ld8(float (&v)[8], const T *p, int i, int step, int n) {
    if constexpr (V) {
        if (i < n) {
            if constexpr (sizeof(T) == 2) {
                const bf16x8 q = *reinterpret_cast<const bf16x8 *>(p + i);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = (float)q[e];
            } else {
                const f32x4 a = *reinterpret_cast<const f32x4 *>(p + i);
                const f32x4 b = *reinterpret_cast<const f32x4 *>(p + i + 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = a[e], v[4 + e] = b[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.f;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (i + e * step < n) ? (float)p[i + e * step] : 0.f;
    }
}

template <typename T, bool V>
__device__ __forceinline__ void st8(const float (&v)[8], T *p, int i, int step, int n) {
    if constexpr (V) {
        if (i >= n) return;
        if constexpr (sizeof(T) == 2) {
            bf16x8 q;
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] = (bf16)v[e];
            *reinterpret_cast<bf16x8 *>(p + i) = q;
        } else {
            *reinterpret_cast<f32x4 *>(p + i) = f32x4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<f32x4 *>(p + i + 4) = f32x4{v[4], v[5], v[6], v[7]};
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (i + e * step < n) p[i + e * step] = (T)v[e];
    }
}

template <typename F>
__device__ __forceinline__ F wave_sum(F v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

// Sum over the W wavefronts of a row; red holds one value per wavefront.
template <int W, typename F>
__device__ __forceinline__ F row_sum(F v, F *red) {
    v = wave_sum(v);
    if constexpr (W > 1) {
        const int w = threadIdx.x >> 6;
        __syncthreads();  // the values of the sum before have been read
        if ((threadIdx.x & 63) == 0) red[w] = v;
        __syncthreads();
        v = 0;
#pragma unroll
        for (int k = 0; k < W; ++k) v += red[k];
    }
    return v;
}

// h (inv + inv_lo) w, rounded once, and to odd: one that is not exact ends in a 1 bit and so lies on
// its own side of every value with fewer bits. Rounded again to such, it gives what the exact product would.
__device__ __forceinline__ float to_odd(float h, float inv, float inv_lo, float w) {
#pragma clang fp contract(off)
    const float p = h * inv, e = __builtin_fmaf(h, inv_lo, __builtin_fmaf(h, inv, -p));
    const float y0 = p * w, f = __builtin_fmaf(e, w, __builtin_fmaf(p, w, -y0));
    const float y = y0 + f, lo = f - (y - y0);
    const uint32_t u = __float_as_uint(y);
    // towards zero, and its last bit set
    const uint32_t odd = (u + (uint32_t)((int)(__float_as_uint(lo) ^ u) >> 31)) | 1u;
    return lo != 0.f ? __uint_as_float(odd) : y;
}

// The codes of 8 values and the scale of their block of 32 (this lane and the
// 3 beside it in its group of 4).
__device__ __forceinline__ void mx_block(const float (&v)[8], u32x2 &codes, uint32_t &scale) {
    uint32_t top = 0;  // largest magnitude as bits: NaN > infinity > every finite value
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
    top = max(top, (uint32_t)__shfl_xor((int)top, 1, 64));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2, 64));
    if (top >= 0x7f800000u) {
        codes = u32x2{0x7f7f7f7fu, 0x7f7f7f7fu};
        scale = 255;
        return;
    }
    // top = 1.m 2^(E-127) <= 1.75 * 2^(p+8): p = E - 135, one more where 1.m > 1.75
    int p = (int)(top >> 23) - 135 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    p = max(p, -127);
    const float inv = __uint_as_float((uint32_t)(127 - p) << 23);  // 2^-p, p in [-127, 120]
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * inv, v[5] * inv, hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * inv, v[7] * inv, hi, true);
    codes = u32x2{(uint32_t)lo, (uint32_t)hi};
    scale = (uint32_t)(p + 127);
}

// TX: storage type of x and y; TR: of the residual. W wavefronts per row, NC
// chunks of 8 values per lane. MX: 8-bit output instead of y.
template <typename TX, typename TR, int W, int NC, bool V, bool MX>
__global__ __launch_bounds__(W > 4 ? W * 64 : kNormThreads) void k_rms_norm(NormArgs a) {
    constexpr int RPB = W > 4 ? 1 : kNormThreads / (64 * W);  // rows per work-group
    using Sum = std::conditional_t<MX, double, float>;
    __shared__ Sum red[W > 1 ? W : 1];
    const int t = threadIdx.x % (64 * W);
    const int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / (64 * W);
    if (r >= a.rows) return;  // only where W == 1: a row per work-group never ends early
    const int n = a.Dg;
    const int64_t at = r * n;
    const TX *x = reinterpret_cast<const TX *>(a.x) + at;
    const TR *res = a.res ? reinterpret_cast<const TR *>(a.res) + at : nullptr;
    const float *wt = a.w + (r % a.groups) * n;
    constexpr int kStep = 64 * W;  // distance of a lane's values where they are taken one by one
    auto first = [&](int c) { return V ? (c * kStep + t) * 8 : c * kStep * 8 + t; };
    float h[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) ld8<TX, V>(h[c], x, first(c), kStep, n);
    if (res) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float q[8];
            ld8<TR, V>(q, res, first(c), kStep, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[c][e] += q[e];
        }
    }
    constexpr bool kLate = W == 16;  // 1024 threads: no registers for the weights, too
    float wv[kLate ? 1 : NC][8];
    if constexpr (!kLate) {
#pragma unroll
        for (int c = 0; c < NC; ++c) ld8<float, V>(wv[c], wt, first(c), kStep, n);
    }
    float sq = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) sq += h[c][e] * h[c][e];
    if (res) {
#pragma unroll
        for (int c = 0; c < NC; ++c) st8<TR, V>(h[c], reinterpret_cast<TR *>(a.res_out) + at, first(c), kStep, n);
    }
    const Sum mean = row_sum<W>((Sum)sq, red) / (Sum)n + (Sum)a.eps;
    const float inv = 1.f / sqrtf((float)mean);
    float inv_lo = 0.f;
    if constexpr (MX) {  // what inv is off by, for to_odd (none where inv is 0 or infinite)
        const double e = 1.0 - mean * inv * inv;
        if (e > -1.0 && e < 1.0) inv_lo = (float)(0.5 * inv * e);
    }
    if (a.rstd && t == 0) a.rstd[r] = inv;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        float y[8];
        if constexpr (kLate) ld8<float, V>(wv[0], wt, first(c), kStep, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (MX) y[e] = to_odd(h[c][e], inv, inv_lo, wv[kLate ? 0 : c][e]);
            else y[e] = h[c][e] * inv * wv[kLate ? 0 : c][e];
        }
        if constexpr (MX) {
            u32x2 codes;
            uint32_t scale;
            mx_block(y, codes, scale);  // every lane: its neighbours read its values
            const int i = first(c);
            if (i < n) {
                *reinterpret_cast<u32x2 *>(a.q + at + i) = codes;
                if ((t & 3) == 0) a.scale[(at + i) >> 5] = (uint8_t)scale;
            }
        } else {
            st8<TX, V>(y, reinterpret_cast<TX *>(a.y) + at, first(c), kStep, n);
        }
    }
}

// y = x in 8 bits (no norm): one chunk of 8 values per lane.
template <typename TX>
__global__ __launch_bounds__(kNormThreads) void k_mx_quantize(const TX *x, uint8_t *q, uint8_t *scale, int64_t n) {
    const int64_t i = ((int64_t)blockIdx.x * kNormThreads + threadIdx.x) * 8;
    float v[8];
    ld8<TX, true>(v, x + (i < n ? i : 0), i < n ? 0 : 8, 0, 8);
    u32x2 codes;
    uint32_t s;
    mx_block(v, codes, s);
    if (i < n) {
        *reinterpret_cast<u32x2 *>(q + i) = codes;
        if ((threadIdx.x & 3) == 0) scale[i >> 5] = (uint8_t)s;
    }
}

// A chunk's 8 values as they are stored.
template <typename T> struct Raw {
    u32x4 q[sizeof(T) / 2];
};
template <typename T, bool V>
__device__ __forceinline__ void ld_raw(Raw<T> &o, const T *p, int i, int step, int n) {
    if constexpr (V) {
#pragma unroll
        for (int c = 0; c < (int)sizeof(T) / 2; ++c)
            o.q[c] = i < n ? reinterpret_cast<const u32x4 *>(p + i)[c] : u32x4{0, 0, 0, 0};
    } else {
        float v[8];
        ld8<T, false>(v, p, i, step, n);
        if constexpr (sizeof(T) == 2) {
            bf16x8 b;
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] = (bf16)v[e];
            o.q[0] = __builtin_bit_cast(u32x4, b);
        } else {
            o.q[0] = __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]});
            o.q[1] = __builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]});
        }
    }
}
template <typename T>
__device__ __forceinline__ void unpack(float (&v)[8], const Raw<T> &r) {
    if constexpr (sizeof(T) == 2) {
        const u32x4 q = r.q[0];
        const bf16x8 b = __builtin_bit_cast(bf16x8, q);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (float)b[e];
    } else {
        const u32x4 q0 = r.q[0], q1 = r.q[1];
        const f32x4 a = __builtin_bit_cast(f32x4, q0), b = __builtin_bit_cast(f32x4, q1);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = a[e], v[4 + e] = b[e];
    }
}

// The gradients, from the stored h and inv. With hh = h inv and g = dy w:
//   dh = inv (g - hh mean(g hh)) + dr_out;   dw = sum over rows of dy hh
// A work-group takes every nb-th row (or 4 rows) of one group (blockIdx.y) and keeps its
// share of dw in registers, lane by lane the columns it reads; the shares are
// added in a fixed order (wavefronts, then work-groups in k_column_sums), so
// the same inputs give the same bits. Bound: HBM. A row's three inputs are
// loaded, as stored, before the row in front of it is finished (kAhead; where
// they fit the registers): a row's time is otherwise its load, the sum over
// the lanes and its store, one after the other (16384 x 1536 in bf16: 201 MB in 45 us,
// 4.5 TB/s; without the loads ahead 61).
template <typename TX, typename TR, int W, int NC, bool V>
__global__ __launch_bounds__(W > 4 ? W * 64 : kNormThreads) void k_rms_norm_bwd(NormBwdArgs a) {
    constexpr int RPB = W > 4 ? 1 : kNormThreads / (64 * W);
    constexpr bool kTwo = sizeof(TX) != sizeof(TR);  // h's gradient in its own type beside x's
    constexpr bool kAhead = W <= 4 && NC * (2 * sizeof(TR) + sizeof(TX)) <= 30;  // 2 rows' inputs: up to 120 registers (8192 x 2048 with an fp32 residual: 4 chunks ahead 64 us, at once 54)
    constexpr bool kTwice = W > 4;  // long rows: the registers hold no row beside dw; it is read again
    constexpr int kStep = 64 * W;
    __shared__ float red[W > 1 ? W : 1];
    __shared__ float share[RPB > 1 ? kStep * NC * 8 : 1];
    const int t = threadIdx.x % kStep, slot = threadIdx.x / kStep;
    const int n = a.Dg, g = blockIdx.y;
    const float *wt = a.w + (int64_t)g * n;
    auto first = [&](int c) { return V ? (c * kStep + t) * 8 : c * kStep * 8 + t; };
    float dw[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[c][e] = 0.f;
    struct Row {
        Raw<TR> h[NC], dr[NC];
        Raw<TX> dy[NC];
        float inv;
    };
    auto load = [&](Row &o, int64_t r) {  // a row behind the last is loaded as zeros
        const bool in = r < a.rows;
        const int64_t at = in ? (r * a.groups + g) * n : 0;
        const int m = in ? n : 0;
        o.inv = in ? a.rstd[r * a.groups + g] : 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            ld_raw<TR, V>(o.h[c], reinterpret_cast<const TR *>(a.h) + at, first(c), kStep, m);
            ld_raw<TX, V>(o.dy[c], reinterpret_cast<const TX *>(a.dy) + at, first(c), kStep, m);
            ld_raw<TR, V>(o.dr[c], reinterpret_cast<const TR *>(a.dres) + at, first(c), kStep, a.dres ? m : 0);
        }
    };
    const int64_t hop = (int64_t)gridDim.x * RPB;
    Row cur, next;
    int64_t r = (int64_t)blockIdx.x * RPB + slot;
    if constexpr (kAhead) load(next, r);
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += hop, r += hop) {
        if constexpr (kAhead) {
            cur = next;
            load(next, r + hop);
        } else if constexpr (!kTwice) {
            load(cur, r);
        } else {
            cur.inv = a.rstd[r * a.groups + g];
        }
        const int64_t at = (r * a.groups + g) * n;
        const int m = r < a.rows ? n : 0;
        const float inv = cur.inv;
        float dot = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float hh[8], dy[8], wv[8];
            if constexpr (kTwice) {
                ld8<TR, V>(hh, reinterpret_cast<const TR *>(a.h) + at, first(c), kStep, n);
                ld8<TX, V>(dy, reinterpret_cast<const TX *>(a.dy) + at, first(c), kStep, n);
            } else {
                unpack(hh, cur.h[c]);
                unpack(dy, cur.dy[c]);
            }
            ld8<float, V>(wv, wt, first(c), kStep, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                hh[e] *= inv;
                dw[c][e] += dy[e] * hh[e];
                dot += dy[e] * wv[e] * hh[e];
            }
        }
        dot = row_sum<W>(dot, red) / (float)n;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float hh[8], dy[8], wv[8], dr[8];
            if constexpr (kTwice) {
                ld8<TR, V>(hh, reinterpret_cast<const TR *>(a.h) + at, first(c), kStep, n);
                ld8<TX, V>(dy, reinterpret_cast<const TX *>(a.dy) + at, first(c), kStep, n);
                ld8<TR, V>(dr, reinterpret_cast<const TR *>(a.dres) + at, first(c), kStep, a.dres ? n : 0);
            } else {
                unpack(hh, cur.h[c]);
                unpack(dy, cur.dy[c]);
                unpack(dr, cur.dr[c]);
            }
            ld8<float, V>(wv, wt, first(c), kStep, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) dr[e] += inv * (dy[e] * wv[e] - hh[e] * inv * dot);
            st8<TX, V>(dr, reinterpret_cast<TX *>(a.dx) + at, first(c), kStep, m);
            if constexpr (kTwo) {
                if (a.dh) st8<TR, V>(dr, reinterpret_cast<TR *>(a.dh) + at, first(c), kStep, m);
            }
        }
    }
    float *part = a.part + ((int64_t)blockIdx.x * a.groups + g) * n;
    if constexpr (RPB > 1) {
        for (int s = 1; s < RPB; ++s) {
            __syncthreads();
            if (slot == s) {
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int e = 0; e < 8; ++e) share[(c * 8 + e) * kStep + t] = dw[c][e];
            }
            __syncthreads();
            if (slot == 0) {
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int e = 0; e < 8; ++e) dw[c][e] += share[(c * 8 + e) * kStep + t];
            }
        }
        if (slot != 0) return;
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) st8<float, V>(dw[c], part, first(c), kStep, n);
}

// out[d] = the nb shares of column d, added by 64 threads, 4 of them in each of 16
// wavefronts, and these in order. One work-group takes 16 columns: its time is a
// chain of nb / 64 loads (1024 x 1536: 4.8 us; 64 columns and 16 threads each: 5.2).
__global__ __launch_bounds__(1024) void k_column_sums(const float *part, float *out, int nb, int64_t D) {
    __shared__ float red[16][16];
    const int c = threadIdx.x & 15, k = threadIdx.x >> 4;
    const int64_t d = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 16 + c;
    float s = 0.f;
    if (d < D) {
#pragma unroll 8
        for (int b = k; b < nb; b += 64) s += part[(int64_t)b * D + d];
    }
    s += __shfl_xor(s, 16, 64);
    s += __shfl_xor(s, 32, 64);
    if ((k & 3) == 0) red[k >> 2][c] = s;
    __syncthreads();
    if (k == 0 && d < D) {
        s = red[0][c];
#pragma unroll
        for (int j = 1; j < 16; ++j) s += red[j][c];
        out[d] = s;
    }
}

ssd_status launch_column_sums(const float *part, float *out, int nb, int64_t D, hipStream_t s) {
    // up to 2^32 columns (65535 groups of 65536): the blocks in rows of 2^20, whose threads stay below kMostThreads
    const int64_t blocks = (D + 15) / 16, x = blocks < (1 << 20) ? blocks : 1 << 20;
    return launch(k_column_sums, dim3((unsigned)x, (unsigned)((blocks + x - 1) / x)), dim3(1024), s, part, out, nb, D) ==
                   hipSuccess
               ? SSD_OK
               : SSD_ERR_HIP;
}

// How a row of n values is spread: wavefronts per row and chunks per lane.
struct NormPlan {
    int W, NC;
};
// One wavefront per row while a row fits 8 chunks a lane (4 where they are taken value by value) and there are rows
// for every SIMD (1024); with fewer rows, 4 wavefronts share one, which
// shortens the chain of a row. Beyond 16384 values 8 or 16 wavefronts take a row.
static NormPlan norm_plan(int64_t rows, int64_t n) {
    if (n > 16384) return {n > 32768 ? 16 : 8, 8};
    const int W = (n <= 512 || (n <= (n % 8 ? 2048 : 4096) && rows >= 1024)) ? 1 : 4;
    const int64_t c = (n + 512 * W - 1) / (512 * W);
    return {W, c <= 4 ? (int)c : 8};
}

template <typename TX, typename TR, bool V, bool MX>
static ssd_status run_norm(const NormArgs &all, hipStream_t s) {
    const NormPlan p = norm_plan(all.rows, all.Dg);
    const int rpb = p.W > 4 ? 1 : kNormThreads / (64 * p.W), threads = p.W > 4 ? 64 * p.W : kNormThreads;
    // rows of one launch, every group of a row among them (65535 at most)
    const int64_t most = kMostThreads / threads * rpb / all.groups * all.groups;
    auto go = [&](auto k) {
        for (int64_t r0 = 0; r0 < all.rows; r0 += most) {
            NormArgs a = all;
            a.rows = all.rows - r0 < most ? all.rows - r0 : most;
            const int64_t at = r0 * all.Dg;
            a.x = static_cast<const TX *>(all.x) + at;
            if (all.res) a.res = static_cast<const TR *>(all.res) + at;
            if (all.res) a.res_out = static_cast<TR *>(all.res_out) + at;
            if constexpr (MX) {
                a.q = all.q + at;
                a.scale = all.scale + at / 32;
            } else {
                a.y = static_cast<TX *>(all.y) + at;
            }
            if (all.rstd) a.rstd = all.rstd + r0;
            if (launch(k, dim3((unsigned)((a.rows + rpb - 1) / rpb)), dim3(threads), s, a) != hipSuccess) return SSD_ERR_HIP;
        }
        return SSD_OK;
    };
    if (p.W == 1) {
        switch (p.NC) {
            case 1: return go(k_rms_norm<TX, TR, 1, 1, V, MX>);
            case 2: return go(k_rms_norm<TX, TR, 1, 2, V, MX>);
            case 3: return go(k_rms_norm<TX, TR, 1, 3, V, MX>);
            case 4: return go(k_rms_norm<TX, TR, 1, 4, V, MX>);
            default: return go(k_rms_norm<TX, TR, 1, 8, V, MX>);
        }
    }
    if (p.W == 4) {
        switch (p.NC) {
            case 1: return go(k_rms_norm<TX, TR, 4, 1, V, MX>);
            case 2: return go(k_rms_norm<TX, TR, 4, 2, V, MX>);
            case 3: return go(k_rms_norm<TX, TR, 4, 3, V, MX>);
            case 4: return go(k_rms_norm<TX, TR, 4, 4, V, MX>);
            default: return go(k_rms_norm<TX, TR, 4, 8, V, MX>);
        }
    }
    return p.W == 8 ? go(k_rms_norm<TX, TR, 8, 8, V, MX>) : go(k_rms_norm<TX, TR, 16, 8, V, MX>);
}

template <typename TX, typename TR>
static ssd_status norm_t(const NormArgs &a, hipStream_t s) {
    if (a.q) return run_norm<TX, TR, true, true>(a, s);
    return a.Dg % 8 == 0 ? run_norm<TX, TR, true, false>(a, s) : run_norm<TX, TR, false, false>(a, s);
}

ssd_status launch_rms_norm(const NormArgs &a, hipStream_t s) {
    if (a.dtype == SSD_F32) return norm_t<float, float>(a, s);
    return a.res_dtype == SSD_F32 ? norm_t<bf16, float>(a, s) : norm_t<bf16, bf16>(a, s);
}

template <typename TX>
static ssd_status run_mx_quantize(const TX *x, uint8_t *q, uint8_t *scale, int64_t n, hipStream_t s) {
    constexpr int64_t most = kMostThreads / kNormThreads * kNormThreads * 8;  // values of one launch
    for (int64_t i = 0; i < n; i += most) {
        const int64_t m = n - i < most ? n - i : most;
        const dim3 grid((unsigned)((m / 8 + kNormThreads - 1) / kNormThreads));
        if (launch(k_mx_quantize<TX>, grid, dim3(kNormThreads), s, x + i, q + i, scale + i / 32, m) != hipSuccess)
            return SSD_ERR_HIP;
    }
    return SSD_OK;
}
ssd_status launch_mx_quantize(const void *x, uint8_t *q, uint8_t *scale, int64_t n, ssd_dtype dtype, hipStream_t s) {
    return dtype == SSD_BF16 ? run_mx_quantize(static_cast<const bf16 *>(x), q, scale, n, s)
                             : run_mx_quantize(static_cast<const float *>(x), q, scale, n, s);
}

// Work-groups per group of columns in the backward: enough to fill the chip
// (1024, 4 to a CU, over all groups), no more than there are rows for.
int norm_bwd_blocks(int64_t rows, int64_t groups, int64_t n) {
    const int rpb = norm_plan(rows, n).W == 1 ? 4 : 1;
    const int64_t most = (rows + rpb - 1) / rpb;
    int64_t want = (1024 + groups - 1) / groups;
    return (int)(want < most ? want : most);
}

template <typename TX, typename TR, bool V>
static ssd_status run_norm_bwd(const NormBwdArgs &a, hipStream_t s) {
    const NormPlan p = norm_plan(a.rows, a.Dg);
    const dim3 grid((unsigned)a.nb, (unsigned)a.groups), block(p.W > 4 ? 64 * p.W : kNormThreads);
    auto go = [&](auto k) { return launch(k, grid, block, s, a) == hipSuccess ? SSD_OK : SSD_ERR_HIP; };
    if (p.W == 1) {
        switch (p.NC) {
            case 1: return go(k_rms_norm_bwd<TX, TR, 1, 1, V>);
            case 2: return go(k_rms_norm_bwd<TX, TR, 1, 2, V>);
            case 3: return go(k_rms_norm_bwd<TX, TR, 1, 3, V>);
            case 4: return go(k_rms_norm_bwd<TX, TR, 1, 4, V>);
            default: return go(k_rms_norm_bwd<TX, TR, 1, 8, V>);
        }
    }
    if (p.W == 4) {
        switch (p.NC) {
            case 1: return go(k_rms_norm_bwd<TX, TR, 4, 1, V>);
            case 2: return go(k_rms_norm_bwd<TX, TR, 4, 2, V>);
            case 3: return go(k_rms_norm_bwd<TX, TR, 4, 3, V>);
            case 4: return go(k_rms_norm_bwd<TX, TR, 4, 4, V>);
            default: return go(k_rms_norm_bwd<TX, TR, 4, 8, V>);
        }
    }
    return p.W == 8 ? go(k_rms_norm_bwd<TX, TR, 8, 8, V>) : go(k_rms_norm_bwd<TX, TR, 16, 8, V>);
}

template <typename TX, typename TR>
static ssd_status norm_bwd_t(const NormBwdArgs &a, hipStream_t s) {
    return a.Dg % 8 == 0 ? run_norm_bwd<TX, TR, true>(a, s) : run_norm_bwd<TX, TR, false>(a, s);
}

ssd_status launch_rms_norm_bwd(const NormBwdArgs &a, hipStream_t s) {
    ssd_status st = a.dtype == SSD_F32         ? norm_bwd_t<float, float>(a, s)
                    : a.res_dtype == SSD_F32 ? norm_bwd_t<bf16, float>(a, s)
                                             : norm_bwd_t<bf16, bf16>(a, s);
    if (st != SSD_OK) return st;
    return launch_column_sums(a.part, a.dw, a.nb, (int64_t)a.Dg * a.groups, s);
}

}  // namespace ssd
