// Matrix products of a layer's projections for gfx950, with the epilogue fused:
//
//   z[m, n] = sum_k x[m, k] w[n, k] + bias[n];   y = act(z) + r[m, n]
//
// from bf16, fp32 or 8-bit operands (e4m3 codes with one power of two for each
// 32 along k; integers with a scale for each row), and the pieces of the backward pass. Sums are fp32 (matrix
// cores; of integers exact, in 32 bits); y is rounded once, at the end, and z once where it is kept.
//
// k_tile: a work-group forms a BM x BN tile of y. A step takes 128 bytes of
// every row of x and w (64 bf16, 32 fp32 or 128 codes): they go straight from
// memory to LDS (16 bytes a lane, no registers), one step ahead of the one
// being multiplied, into the other of two buffers. A row's 8 chunks of 16
// bytes lie at chunk ^ (row % 8), so that the 8 rows that one LDS cycle reads
// lie in different banks; since the loads write LDS in lane order, the lanes
// permute the addresses they load from. Lane l = 16 kg + r takes chunks kg and
// kg + 4 of its row: that is the order of k that the 8-bit product's scales
// imply (lane kg's scale is that of k in [32 kg, 32 kg + 32)), and any order
// does for the other types as long as x and w share it. The 8-bit product
// (twice the bf16 rate) adds 8 consecutive k in fixed point, 13 bits below the
// largest of the 8 products, and everything else in fp32: measured on random
// codes, 2^-15.7 of the sum of magnitudes on average, some 1e-4 of a result at
// in = 2048, where the codes' own rounding is 2.6e-2. Products in bf16 (every
// code is a bf16) would be exact at half the rate.
//
// fp32 operands are split, as they are read from LDS, into three bf16 each, and
// six of the nine products formed: 1.3 times the rate of the fp32 matrix cores
// (8192 x 4096 x 2048: 660 us, 208 TFLOP/s; the library's fp32 product 151).
//
// The product is formed as w x^T, so that a lane holds 4 consecutive n of one
// row; the epilogue turns 16 x (columns of a wavefront) at a time through LDS
// into whole lines of rows.
//
// Bound: the matrix cores and the waits for their operands. Microseconds on a warm GPU, bf16, operands that
// change from call to call, the library's plain product beside it: 8192 x 4096 x 2048 113 (90), with a residual
// 135; 8192 x 2048 x 8512 263 (250); 16384 x 768 x 3352 99 (133); 64 x 2048 x 8512 13.5 (19.5); 8192 x 8192 x 8192
// 814 (697); 8 bits 8192 x 2048 x 8512 149 to 166. The matrix cores are busy 52% of the cycles of the first (42% with
// the residual, 37% in 8 bits), and 70% of those that another 4096 along k add to it (87% where the
// operands stay in the last-level cache). The rest of a round of tiles is its start and its epilogue, where nothing is
// multiplied, 10 to 14 us, and the residual's way from memory. Measured and left: 4
// wavefronts a tile, 32 x 32 matrix instructions, a wave priority around the
// products, loads two steps ahead (all within 2% or slower).
//
// k_skinny (up to 16 rows, decoding): the time is one read of w. A
// work-group takes 16 rows of w, its 8 wavefronts split k, and both operands
// go from memory to the matrix cores' registers; the 8 shares are added
// through LDS. 8 x 2048 x 8512 in bf16 (35 MB): 12 us, 2.9 TB/s, of which the
// launch and the first loads are half; 1 x 2048 x 50257 (206 MB): 40 us, 5.1 TB/s.
// 4 or 16 wavefronts, and loads past the caches, were slower.
#include <type_traits>

#include "ssd_common.h"
#include "ssd_internal.h"

namespace ssd {

constexpr int kBF16 = 0, kF32 = 1, kMX = 2, kInt = 3;
constexpr int kParts = 3;  // beside the activations
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;

// 16 (4) bytes a lane from base + voff + soff, zeros behind `bytes`, to consecutive places from dst on.
__device__ __forceinline__ void to_lds16(const void *base, uint32_t bytes, void *dst, uint32_t voff, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(base, bytes), (lds_void *)dst, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void to_lds4(const void *base, uint32_t bytes, void *dst, uint32_t voff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(base, bytes), (lds_void *)dst, 4, voff, 0, 0, 0);
}

// fp32 in three bf16: x = a + b + c exactly (8 bits of the 24-bit mantissa each, cut off, not
// rounded). A product of two such sums keeps a a', a b', b a', b b', a c' and c a': the
// three that are left out are under 2^-21 of it, 2^-24 on average.
struct Split {
    bf16x8 a, b, c;
};
__device__ __forceinline__ Split split8(u32x4 l, u32x4 h) {
    uint32_t a[4], b[4], c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = i < 2 ? l[2 * i] : h[2 * i - 4], v = i < 2 ? l[2 * i + 1] : h[2 * i - 3];
        const float ru = __uint_as_float(u) - __uint_as_float(u & 0xffff0000u);
        const float rv = __uint_as_float(v) - __uint_as_float(v & 0xffff0000u);
        const uint32_t ub = __float_as_uint(ru), vb = __float_as_uint(rv);
        const uint32_t uc = __float_as_uint(ru - __uint_as_float(ub & 0xffff0000u));
        const uint32_t vc = __float_as_uint(rv - __uint_as_float(vb & 0xffff0000u));
        a[i] = __builtin_amdgcn_perm(v, u, 0x07060302u);  // the upper halves of u and v
        b[i] = __builtin_amdgcn_perm(vb, ub, 0x07060302u);
        c[i] = __builtin_amdgcn_perm(vc, uc, 0x07060302u);
    }
    return {__builtin_bit_cast(bf16x8, u32x4{a[0], a[1], a[2], a[3]}), __builtin_bit_cast(bf16x8, u32x4{b[0], b[1], b[2], b[3]}),
            __builtin_bit_cast(bf16x8, u32x4{c[0], c[1], c[2], c[3]})};
}
__device__ __forceinline__ f32x4 mma_split(const Split &w, const Split &x, f32x4 acc) {  // small terms first
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.c, x.a, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.a, x.c, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.b, x.b, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.b, x.a, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.a, x.b, acc, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.a, x.a, acc, 0, 0, 0);
}

// Schedules R LDS reads one by one between the first of P matrix-core
// instructions, and V loads between the rest.
template <int R, int P, int V>
__device__ __forceinline__ void mix() {
    constexpr int each = (R + P - 1) / P, n = (R + each - 1) / each;
#pragma unroll
    for (int i = 0; i < n; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, each, 0);
    }
    constexpr int left = P > n ? P - n : 1, per = (V + left - 1) / left;
#pragma unroll
    for (int i = 0; i < left && V > 0; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x010, per, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
}

// Where chunk c of row k lies in a row of CPR chunks (rows along k), and which chunk lies at place p.
template <int CPR>
__device__ __forceinline__ int swizzled(int c, int k) {
    if constexpr (CPR == 8) return c ^ (((k >> 1) & 1) * 2 | ((k >> 3) & 1) * 4);
    const int q = (c ^ (2 * (k & 3))) + 8 * ((k >> 3) & 1);
    return q >= CPR ? q - CPR : q;
}
template <int CPR>
__device__ __forceinline__ int unswizzled(int p, int k) {
    if constexpr (CPR == 8) return swizzled<8>(p, k);
    const int q = p - 8 * ((k >> 3) & 1);
    return (q < 0 ? q + CPR : q) ^ (2 * (k & 3));
}

// Every wavefront's loads into LDS have arrived (a barrier alone does not wait
// for them), and its reads too.
__device__ __forceinline__ void arrive() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __syncthreads();
}

// 4 consecutive rows of one column a lane: in each group of 16, lane j gives the
// address of 8 bytes of row j / 4 and receives the column of its own number.
__device__ __forceinline__ u32x2 lds_transposed(const char *p) {
    typedef short v4i16 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) v4i16 lds_v4i16;
    const v4i16 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)p);
    return __builtin_bit_cast(u32x2, v);
}

// 128 bytes (lane's 2 x 16) of a row of w against those of a row of x.
template <int KIND>
__device__ __forceinline__ f32x4 mma2(u32x4 wl, u32x4 wh, u32x4 xl, u32x4 xh, f32x4 c, int sw, int sx) {
    if constexpr (KIND == kBF16) {
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wl), __builtin_bit_cast(bf16x8, xl), c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wh), __builtin_bit_cast(bf16x8, xh), c, 0, 0, 0);
    } else if constexpr (KIND == kF32) {
        const f32x4 a = __builtin_bit_cast(f32x4, wl), b = __builtin_bit_cast(f32x4, xl);
        const f32x4 d = __builtin_bit_cast(f32x4, wh), e = __builtin_bit_cast(f32x4, xh);
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(d[i], e[i], c, 0, 0, 0);
    } else if constexpr (KIND == kInt) {  // the accumulators' bits are integers
        i32x4 d = __builtin_bit_cast(i32x4, c);
        d = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, wl), __builtin_bit_cast(i32x4, xl), d, 0, 0, 0);
        d = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, wh), __builtin_bit_cast(i32x4, xh), d, 0, 0, 0);
        c = __builtin_bit_cast(f32x4, d);
    } else {
        typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));
        const u32x8 w = __builtin_shufflevector(wl, wh, 0, 1, 2, 3, 4, 5, 6, 7);
        const u32x8 x = __builtin_shufflevector(xl, xh, 0, 1, 2, 3, 4, 5, 6, 7);
        c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(i32x8, w), __builtin_bit_cast(i32x8, x),
                                                             c, 0, 0, 0, sw, 0, sx);
    }
    return c;
}

// The activations and their slopes (act: a constant where they are called). kFast, for values that are
// rounded to bf16: the vector unit's 2^x and 1/x (1 ulp each), and for GELU
//   erfc(u) = (a1 t + .. + a7 t^7) e^(-u^2),  t = 1 / (1 + 0.505 u),  u >= 0
// whose exponential the slope needs, too. The form is Abramowitz and Stegun's (7.1.26); its 5 terms are
// off by 1.5e-7 of 1, which far from zero is 4% of erfc. These 7 were fitted (least largest error, weighted)
// to stay within 1.2e-7 of 1 and within 2^-13 of erfc itself for all u: a GELU of z = -12 is as good as one of -1.
// expf, erff and a division took k_dz from memory's time to the vector unit's. In fp32 erfc, not 1 + erf, which
// has nothing left below z = -5.5.
template <bool kFast>
__device__ __forceinline__ float sigmoid(float z) {
    if constexpr (kFast) return __builtin_amdgcn_rcpf(1.f + fast_exp2(-kLog2e * z));
    return 1.f / (1.f + expf(-z));
}
// erfc(-z / sqrt 2) / 2, and e^(-z^2 / 2)
template <bool kFast>
__device__ __forceinline__ float normal_cdf(float z, float &e) {
    if constexpr (kFast) {
        e = fast_exp2(-0.5f * kLog2e * z * z);
        const float t = __builtin_amdgcn_rcpf(1.f + 0.505f * 0.70710678f * fabsf(z));
        const float c = 0.5f * e * t * (0.284915149f + t * (0.283997625f + t * (0.264520407f + t * (0.0839478597f +
                        t * (0.328074515f + t * (-0.329984188f + t * 0.0845286995f))))));
        return z < 0.f ? c : 1.f - c;
    }
    e = expf(-0.5f * z * z);
    return 0.5f * erfcf(z * -0.70710678118654752f);
}
template <bool kFast>
__device__ __forceinline__ float act_of(float z, int act) {
    if (act == SSD_ACT_SILU) return kFast ? z * sigmoid<true>(z) : z / (1.f + expf(-z));
    float e;
    if (act == SSD_ACT_GELU) return z * normal_cdf<kFast>(z, e);
    return z;
}
template <bool kFast>
__device__ __forceinline__ float act_slope(float z, int act) {
    if (act == SSD_ACT_SILU) {
        const float g = sigmoid<kFast>(z);
        return g * (1.f + z * (1.f - g));
    }
    if (act == SSD_ACT_GELU) {
        float e;
        const float c = normal_cdf<kFast>(z, e);
        return c + z * 0.3989422804014327f * e;
    }
    return 1.f;
}

template <typename TO>
__device__ __forceinline__ void put4(TO *p, const float (&v)[4], int n, bool whole) {
    if (whole) {
        if constexpr (sizeof(TO) == 2) {
            *reinterpret_cast<bf16x4 *>(p) = bf16x4{(bf16)v[0], (bf16)v[1], (bf16)v[2], (bf16)v[3]};
        } else {
            *reinterpret_cast<f32x4 *>(p) = f32x4{v[0], v[1], v[2], v[3]};
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = (TO)v[i];
    }
}

template <typename TO>
__device__ __forceinline__ void get4(float (&v)[4], const TO *p, int n, bool whole) {
    if (whole) {
        if constexpr (sizeof(TO) == 2) {
            const bf16x4 q = *reinterpret_cast<const bf16x4 *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = (float)q[i];
        } else {
            const f32x4 q = *reinterpret_cast<const f32x4 *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = q[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < n ? (float)p[i] : 0.f;
    }
}

// The epilogue of 4 consecutive columns n .. n + 3 of row m, with their bias
// and residual (zeros where there is none) already loaded. kWhole: N and
// the rows' stride are multiples of 4, so every group of 4 is whole and aligned.
template <typename TO, int ACT, bool kWhole>
__device__ __forceinline__ void finish4(const LinearArgs &a, int m, int n, float (&v)[4], const float (&bias)[4],
                                        const float (&res)[4]) {
    const int left = a.N - n;
    if (m >= a.M || left <= 0) return;
    const int64_t at = (int64_t)m * a.ldy + n;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += bias[i];
    if (a.pre) put4<TO>(reinterpret_cast<TO *>(a.pre) + at, v, left, kWhole);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = act_of<sizeof(TO) == 2>(v[i], ACT) + res[i];
    put4<TO>(reinterpret_cast<TO *>(a.y) + at, v, left, kWhole);
}
__device__ __forceinline__ void bias4(const LinearArgs &a, int n, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (a.bias && n + i < a.N) ? a.bias[n + i] : 0.f;
}
// Integers: the scales of row m and of 4 consecutive columns, and sums with them.
__device__ __forceinline__ float row_scale(const LinearArgs &a, int m) { return m < a.M ? a.xs[m] : 0.f; }
__device__ __forceinline__ void column_scales4(const LinearArgs &a, int n, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = n + i < a.N ? a.ws[n + i] : 0.f;
}
// The sum goes by the row's scale first, but where that may be beyond 2^127: sums are at most 2^31, so what is infinite then
// is so with both scales (and nothing is lost below: the product of an integer and a number has its places).
__device__ __forceinline__ bool far(float xs) { return fabsf(xs) > 0x1p96f; }
__device__ __forceinline__ float scaled(float bits, float xs, float ws) {
    return (float)__float_as_int(bits) * (far(xs) ? ws : xs) * (far(xs) ? xs : ws);
}
// A branch: to choose value by value took 3% longer (8192 x 2048 x 8512: 162 us, 168 so).
__device__ __forceinline__ void scale4(float xs, const float (&ws)[4], float (&v)[4]) {
    if (__builtin_expect(__any(far(xs)), 0)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = scaled(v[i], xs, ws[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)__float_as_int(v[i]) * xs * ws[i];
    }
}
__device__ __forceinline__ float add_bits(float a, float b) { return __int_as_float(__float_as_int(a) + __float_as_int(b)); }
template <int KIND>
__device__ __forceinline__ void scale4_any(const LinearArgs &a, int m, int n, float (&v)[4]) {
    if constexpr (KIND == kInt) {
        float ws[4];
        column_scales4(a, n, ws);
        scale4(row_scale(a, m), ws, v);
    }
}
template <typename TO, bool kWhole>
__device__ __forceinline__ void res4(const LinearArgs &a, int m, int n, float (&v)[4]) {
    if (a.res && m < a.M && n < a.N) {
        get4<TO>(v, reinterpret_cast<const TO *>(a.res) + (int64_t)m * a.ldy + n, a.N - n, kWhole);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = 0.f;
    }
}
// 4 columns of the residual as stored (whole groups), zeros where there is none.
template <typename TO>
struct Res {
    uint32_t w[sizeof(TO)];
    __device__ __forceinline__ void load(const LinearArgs &a, int m, int n) {
        typedef uint32_t word __attribute__((ext_vector_type(sizeof(TO))));
        word q = {};
        if (a.res && m < a.M && n < a.N) q = *reinterpret_cast<const word *>(reinterpret_cast<const TO *>(a.res) + (int64_t)m * a.ldy + n);
#pragma unroll
        for (int k = 0; k < (int)sizeof(TO); ++k) w[k] = q[k];
    }
    __device__ __forceinline__ void get(float (&v)[4]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = __uint_as_float(sizeof(TO) == 4 ? w[e % sizeof(TO)] : e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
    }
};
// Everything for one group of 4.
template <typename TO>
__device__ __forceinline__ void finish4_any(const LinearArgs &a, int m, int n, float (&v)[4]) {
    float bias[4], res[4];
    bias4(a, n, bias);
    auto go = [&](auto whole) {
        constexpr bool kWhole = decltype(whole)::value;
        res4<TO, kWhole>(a, m, n, res);
        if (a.act == SSD_ACT_SILU) finish4<TO, SSD_ACT_SILU, kWhole>(a, m, n, v, bias, res);
        else if (a.act == SSD_ACT_GELU) finish4<TO, SSD_ACT_GELU, kWhole>(a, m, n, v, bias, res);
        else finish4<TO, SSD_ACT_NONE, kWhole>(a, m, n, v, bias, res);
    };
    if (a.whole) go(std::true_type{});
    else go(std::false_type{});
}

// The values of 16 bytes of a row that lie before its end, zeros behind it.
template <typename T>
__device__ __forceinline__ u32x4 ld_rest(const char *row, uint32_t off, uint32_t end) {
    constexpr int E = 16 / (int)sizeof(T);
    union {
        T e[E];
        u32x4 v;
    } q;
#pragma unroll
    for (int i = 0; i < E; ++i) q.e[i] = off + i * sizeof(T) < end ? *reinterpret_cast<const T *>(row + off + i * sizeof(T)) : (T)0.f;
    return q.v;
}

// Tile number of a work-group: consecutive ones on one XCD (work-groups are
// dealt to the 8 XCDs in turn), walked down columns of 8 tiles of m, so that
// an XCD's L2 sees few rows of x and w at a time.
__device__ __forceinline__ void tile_of(int id, int nm, int nn, int &tm, int &tn) {
    const int total = nm * nn, per = total >> 3, more = total & 7;
    const int xcd = id & 7, k = id >> 3;
    const int t = xcd * per + (xcd < more ? xcd : more) + k;
    constexpr int G = 8;
    const int band = t / (G * nn), in = t - band * G * nn;
    const int rows = min(G, nm - band * G);
    tm = band * G + in % rows;
    tn = in / rows;
}

// EPI: the activation, or kParts to store the fp32 parts of a split sum.
// XT, WT (bf16): x or w is given with its rows along k (k x M, k x N), as the
// backward pass has them. A step then takes 64 rows of BM (BN) columns, and
// the lanes' 8 values along k are read down the columns with LDS's transposing
// read. 32 of its lanes take 32 bytes of rows k .. k + 3 and k + 8 .. k + 11 each;
// the chunks of a row are moved by swizzled() so that these 8 pieces of 32 bytes lie in
// different banks (without the second four: half of the reads' cycles were conflicts).
template <int KIND, typename TO, int BM, int BN, int WM, int WN, int EPI, bool XT, bool WT, bool RAGGED>
__global__ __launch_bounds__(64 * WM * WN, BM == 64 ? 4 : 2) void k_tile(LinearArgs a) {
    constexpr int NW = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;  // loads per wavefront and step, 8 rows each
    static_assert(LA * 8 * NW == BM && LB * 8 * NW == BN, "rows divide over the wavefronts");
    static_assert(KIND != kMX || (BM % 64 == 0 && BN % 64 == 0 && BM + BN <= 64 * NW), "one load of scales per wavefront and step");
    static_assert(KIND == kBF16 || (!XT && !WT), "the transposing read is of 16 bits");
    // one array per buffer: the compiler then knows that reads of one do not wait for the loads into the other
    __shared__ __attribute__((aligned(128))) char s0[(BM + BN) * 128];
    __shared__ __attribute__((aligned(128))) char s1[(BM + BN) * 128];
    __shared__ __attribute__((aligned(16))) uint8_t q0[KIND == kMX ? 256 * NW : 16];
    __shared__ __attribute__((aligned(16))) uint8_t q1[KIND == kMX ? 256 * NW : 16];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int r = lane & 15, kg = lane >> 4;
    int tm, tn;
    tile_of(blockIdx.x, a.nm, a.nn, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    // A load takes 8 rows; each has a resource of its own that ends with the operand, so that one
    // offset per lane serves all. Loads whole behind the operand take its first 8 rows of this tile
    // instead: their rows of y are not stored.
    const char *xrow[LA], *wrow[LB];
    uint32_t xlen[LA], wlen[LB], xoff[LA], woff[LB];
    // this lane's chunk of the 8 rows of a load
    const uint32_t chunk = (uint32_t)(((lane & 7) ^ (lane >> 3)) << 4);
    const uint32_t va = (uint32_t)(lane >> 3) * (uint32_t)a.ldx + chunk, vb = (uint32_t)(lane >> 3) * (uint32_t)a.ldw + chunk;
#pragma unroll
    for (int j = 0; j < LA; ++j) {
        if constexpr (XT) {
            const int g = (w * LA + j) * 64 + lane, k = g / (BM / 8), c = g % (BM / 8);
            xoff[j] = (uint32_t)k * (uint32_t)a.ldx + (uint32_t)(unswizzled<BM / 8>(c, k) << 4);
        } else {
            int row = m0 + (w * LA + j) * 8;
            row = row < a.M ? row : m0;
            xrow[j] = reinterpret_cast<const char *>(a.x) + (int64_t)row * a.ldx;
            xlen[j] = (uint32_t)(min(8, a.M - row) * a.ldx);
        }
    }
#pragma unroll
    for (int j = 0; j < LB; ++j) {
        if constexpr (WT) {
            const int g = (w * LB + j) * 64 + lane, k = g / (BN / 8), c = g % (BN / 8);
            woff[j] = (uint32_t)k * (uint32_t)a.ldw + (uint32_t)(unswizzled<BN / 8>(c, k) << 4);
        } else {
            int row = n0 + (w * LB + j) * 8;
            row = row < a.N ? row : n0;
            wrow[j] = reinterpret_cast<const char *>(a.w) + (int64_t)row * a.ldw;
            wlen[j] = (uint32_t)(min(8, a.N - row) * a.ldw);
        }
    }
    const uint8_t *srow = nullptr;
    uint32_t slen = 0, vs = 0;
    if constexpr (KIND == kMX) {
        // scales: wavefronts below BM / 64 take rows of x, the others rows of w; 4 bytes a row and step
        const bool of_x = w < BM / 64;
        const int row0 = of_x ? m0 + w * 64 : n0 + (w - BM / 64) * 64, most = of_x ? a.M : a.N;
        const int64_t rows = w < (BM + BN) / 64 ? max(0, min(64, most - row0)) : 0;
        const uint8_t *p = (of_x ? a.xscale + (int64_t)row0 * a.lds : a.wscale + (int64_t)row0 * a.lds);
        srow = rows > 0 ? p : a.xscale;
        slen = (uint32_t)(rows * a.lds);
        vs = (uint32_t)lane * (uint32_t)a.lds;
    }
    const int per = a.steps_per_split, first = (int)blockIdx.y * per;
    const int steps = min(per, a.steps - first);

    auto fetch = [&](int s, char *buf, uint8_t *sc) {
        // a step behind the last loads zeros, and so do the chunks behind the row's end where the last
        // ends inside its 128 bytes. Only k0, which lies inside every range, goes into the scalar offset:
        // that one is subtracted from the range before the comparison
        const bool live = s < steps;
        const uint32_t k0 = live ? (uint32_t)(first + s) * 128u : 0u;
        const uint32_t off = oob_if(!live || k0 + chunk >= a.kbytes, 0);
        // rows along k: the 64 rows of the step, from the tile's first column on; zeros behind the last row
        const int k1 = (int)(k0 >> 1);
        const int rows = max(0, live ? min(64, a.krows - k1) : 0);
        const char *xt = nullptr, *wt = nullptr;
        uint32_t xtl = 0, wtl = 0;
        if constexpr (XT) {
            xt = reinterpret_cast<const char *>(a.x) + (int64_t)k1 * a.ldx + m0 * 2;
            xtl = (uint32_t)max(0, rows * (int)a.ldx - m0 * 2);
        }
        if constexpr (WT) {
            wt = reinterpret_cast<const char *>(a.w) + (int64_t)k1 * a.ldw + n0 * 2;
            wtl = (uint32_t)max(0, rows * (int)a.ldw - n0 * 2);
        }
#pragma unroll
        for (int j = 0; j < LA; ++j) {
            char *to = buf + (w * LA + j) * 1024;
            if constexpr (XT) to_lds16(xt, xtl, to, xoff[j], 0);
            else to_lds16(xrow[j], xlen[j], to, va | off, k0);
        }
#pragma unroll
        for (int j = 0; j < LB; ++j) {
            char *to = buf + BM * 128 + (w * LB + j) * 1024;
            if constexpr (WT) to_lds16(wt, wtl, to, woff[j], 0);
            else to_lds16(wrow[j], wlen[j], to, vb | off, k0);
        }
        if constexpr (KIND == kMX)
            to_lds4(srow, slen, sc + w * 256, (vs + (uint32_t)(first + s) * 4u) | oob_if(!live, 0));
    };

    // RAGGED: rows end inside 16 bytes (their starts are multiples of 4 only). The chunk that they end in
    // brings the next row's first values along. It is written once more, value by value, in the step that has it.
    // (777 x 1003 x 515 in fp32 27.2 us with copies in whole chunks in front, 21.7 so; 8192 x 4094 x 2048 in bf16
    // 138 and 117. A kernel of its own: the branch in a step costs 8192 x 4096 x 2048 1.5%)
    int ragged = a.steps - 1 - first;
    if (ragged >= steps) ragged = -1;  // another split's
    auto mend = [&](char *buf) {
        for (int t = (int)threadIdx.x; t < BM + BN; t += 64 * NW) {
            const bool of_x = t < BM;
            const int row = of_x ? m0 + t : n0 + t - BM;
            if (row >= (of_x ? a.M : a.N)) continue;
            const char *p = reinterpret_cast<const char *>(of_x ? a.x : a.w) + (int64_t)row * (of_x ? a.ldx : a.ldw);
            const int c = (int)(a.kbytes >> 4) & 7;
            *reinterpret_cast<u32x4 *>(buf + t * 128 + ((c ^ (t & 7)) << 4)) = ld_rest<TO>(p, a.kbytes & ~15u, a.kbytes);
        }
        __syncthreads();
    };

    const int wm = w / WN, wn = w % WN;
    const int pa = (wm * TM * 16 + r) * 128 + ((kg ^ (r & 7)) << 4);       // chunk kg of row r; kg + 4 is at ^ 64
    const int pb = (BM + wn * TN * 16 + r) * 128 + ((kg ^ (r & 7)) << 4);
    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // A step's products go in NQ parts, TQ of the wavefront's row blocks each. The
    // operands of a part are read while the part before it is multiplied: the first
    // part of the next step (and its w) during this step's last, right behind the
    // barrier, so that the matrix cores have work across it.
    constexpr int NQ = (KIND == kMX || TM < 4) ? TM : 4, TQ = TM / NQ;  // 8 bits: registers for the scales, too
    static_assert(TQ * NQ == TM && NQ % 2 == 0, "parts of a step");
    constexpr int kMma = (KIND == kBF16 || KIND == kInt) ? 2 : KIND == kF32 ? 6 : 1;  // matrix-core instructions of a product
    constexpr int kReadsX = TQ * (XT ? 4 : KIND == kMX ? 3 : 2), kReadsW = TN * (WT ? 4 : KIND == kMX ? 3 : 2);
    struct WRegs {
        u32x4 l[TN], h[TN];
        int s[TN];
    } w0, w1;
    struct XRegs {
        u32x4 l[TQ], h[TQ];
        int s[TQ];
    } x0, x1;
    // rows along k: this lane's 8 bytes of rows 8 kg + r / 4 and on, at block b of 16 columns
    const int tk = 8 * kg + (r >> 2), tc = (r >> 1) & 1, th = (r & 1) * 8;
    auto down = [&](u32x4 &l, u32x4 &h, const char *part, int b, auto chunks) {
        constexpr int CPR = decltype(chunks)::value, width = CPR * 16;
        // 4 and 32 rows on the chunk lies at the same place; in rows of 8 chunks, too
        const char *p = part + tk * width + (swizzled<CPR>(2 * b + tc, tk) << 4) + th;
        const u32x2 l0 = lds_transposed(p), l1 = lds_transposed(p + 4 * width);
        const u32x2 h0 = lds_transposed(p + 32 * width), h1 = lds_transposed(p + 36 * width);
        l = __builtin_shufflevector(l0, l1, 0, 1, 2, 3);
        h = __builtin_shufflevector(h0, h1, 0, 1, 2, 3);
    };
    auto read_w = [&](WRegs &f, const char *buf, const uint8_t *sc) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            f.s[j] = 0;
            if constexpr (WT) {
                down(f.l[j], f.h[j], buf + BM * 128, wn * TN + j, std::integral_constant<int, BN / 8>{});
                continue;
            }
            f.l[j] = *reinterpret_cast<const u32x4 *>(buf + pb + j * 2048);
            f.h[j] = *reinterpret_cast<const u32x4 *>(buf + (pb ^ 64) + j * 2048);
            f.s[j] = KIND == kMX ? sc[(BM + (wn * TN + j) * 16 + r) * 4 + kg] : 0;
        }
    };
    auto read_x = [&](XRegs &f, const char *buf, const uint8_t *sc, int q) {
#pragma unroll
        for (int i = 0; i < TQ; ++i) {
            f.s[i] = 0;
            if constexpr (XT) {
                down(f.l[i], f.h[i], buf, wm * TM + q * TQ + i, std::integral_constant<int, BM / 8>{});
                continue;
            }
            f.l[i] = *reinterpret_cast<const u32x4 *>(buf + pa + (q * TQ + i) * 2048);
            f.h[i] = *reinterpret_cast<const u32x4 *>(buf + (pa ^ 64) + (q * TQ + i) * 2048);
            f.s[i] = KIND == kMX ? sc[((wm * TM + q * TQ + i) * 16 + r) * 4 + kg] : 0;
        }
    };
    Split ws[KIND == kF32 ? TN : 1];
    auto multiply = [&](const WRegs &wf, const XRegs &xf, int q) {
        if constexpr (KIND == kF32) {
            if (q == 0) {
#pragma unroll
                for (int j = 0; j < TN; ++j) ws[j] = split8(wf.l[j], wf.h[j]);
            }
#pragma unroll
            for (int i = 0; i < TQ; ++i) {
                const Split xs = split8(xf.l[i], xf.h[i]);
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[q * TQ + i][j] = mma_split(ws[j], xs, acc[q * TQ + i][j]);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < TQ; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[q * TQ + i][j] = mma2<KIND>(wf.l[j], wf.h[j], xf.l[i], xf.h[i], acc[q * TQ + i][j], wf.s[j], xf.s[i]);
    };
    auto step = [&](int s, char *buf, uint8_t *sc, char *nbuf, uint8_t *nsc, WRegs &wf, WRegs &nwf) {
#pragma unroll
        for (int q = 0; q < NQ - 1; ++q) {
            read_x((q & 1) ? x0 : x1, buf, sc, q + 1);
            multiply(wf, (q & 1) ? x1 : x0, q);
            mix<kReadsX, TQ * TN * kMma, 0>();  // the compiler would move every read down to its first use
        }
        arrive();  // step s + 1 is there, and everybody has read all of step s
        if (RAGGED && s + 1 == ragged) mend(nbuf);
        __builtin_amdgcn_sched_barrier(0);
        read_w(nwf, nbuf, nsc);
        read_x(x0, nbuf, nsc, 0);
        fetch(s + 2, buf, sc);
        multiply(wf, x1, NQ - 1);
        // between the products, too: in front of them the matrix cores would wait for 8 wavefronts' reads
        mix<kReadsW + kReadsX, TQ * TN * kMma, LA + LB>();
    };

    // pairs of steps, without a branch: the accumulators then stay where they are
    fetch(0, s0, q0);
    arrive();
    if (RAGGED && ragged == 0) mend(s0);
    fetch(1, s1, q1);
    read_w(w0, s0, q0);
    read_x(x0, s0, q0, 0);
    for (int s = 0; s < steps; s += 2) {
        step(s, s0, q0, s1, q1, w0, w1);
        step(s + 1, s1, q1, s0, q0, w1, w0);
    }
    arrive();

    // epilogue: 16 rows of the wavefront's columns at a time through LDS
    constexpr int CW = TN * 16, LDC = CW + 4;
    static_assert(NW * 16 * LDC * 4 <= (BM + BN) * 128, "the wavefronts' pieces fit one buffer");
    float *piece = reinterpret_cast<float *>(s0) + w * 16 * LDC;
    // a lane's group of 4 columns in pass p over the 16 rows
    constexpr int LPR = CW / 4, NP = CW / 16;
    const int mw = m0 + wm * TM * 16, nw = n0 + wn * CW;
    auto row_of = [&](int p) { return (p * 64 + lane) / LPR; };
    auto col_of = [&](int p) { return ((p * 64 + lane) % LPR) * 4; };
    auto stage = [&](int i) {
#pragma unroll
        for (int j = 0; j < TN; ++j) *reinterpret_cast<f32x4 *>(piece + r * LDC + j * 16 + kg * 4) = acc[i][j];
        __builtin_amdgcn_wave_barrier();
    };
    auto staged = [&](int p, float (&v)[4]) {
        const f32x4 c = *reinterpret_cast<const f32x4 *>(piece + row_of(p) * LDC + col_of(p));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = c[e];
    };
    if constexpr (EPI == kParts) {
        const bool whole = (a.N & 3) == 0;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            stage(i);
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                float v[4];
                staged(p, v);
                const int m = mw + i * 16 + row_of(p), n = nw + col_of(p);
                if (m < a.M && n < a.N) put4<float>(a.part + blockIdx.y * part_stride(a.M, a.N) + (int64_t)m * a.N + n, v, a.N - n, whole);
            }
            __builtin_amdgcn_wave_barrier();
        }
        return;
    }
    if (EPI == SSD_ACT_NONE && a.whole) {
        // the next rows' residual is on its way while 16 rows are finished: 48 rows of it in bf16 (8192 x 2048 x 8512
        // from integers, with a residual, 211 us; with 16 rows 251), 16 in fp32. The backward pass has none.
        constexpr int AHEAD = sizeof(TO) == 2 && !XT && !WT ? 3 : 1;
        float bias[NP][4], ws[KIND == kInt ? NP : 1][4], xs[2][KIND == kInt ? NP : 1];
        Res<TO> res[AHEAD + 1][NP];
        auto ask = [&](int i) {
#pragma unroll
            for (int p = 0; p < NP; ++p) res[i % (AHEAD + 1)][p].load(a, mw + i * 16 + row_of(p), nw + col_of(p));
        };
#pragma unroll
        for (int i = 0; i < AHEAD && i < TM; ++i) ask(i);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            if constexpr (KIND == kInt) {
                column_scales4(a, nw + col_of(p), ws[p]);
                xs[0][p] = row_scale(a, mw + row_of(p));
            }
            bias4(a, nw + col_of(p), bias[p]);
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            stage(i);
            if (i + AHEAD < TM) ask(i + AHEAD);
            if constexpr (KIND == kInt) {
#pragma unroll
                for (int p = 0; p < NP; ++p)
                    if (i + 1 < TM) xs[(i + 1) & 1][p] = row_scale(a, mw + (i + 1) * 16 + row_of(p));
            }
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                float v[4], r4[4];
                staged(p, v);
                res[i % (AHEAD + 1)][p].get(r4);
                if constexpr (KIND == kInt) scale4(xs[i & 1][p], ws[p], v);
                finish4<TO, SSD_ACT_NONE, true>(a, mw + i * 16 + row_of(p), nw + col_of(p), v, bias[p], r4);
            }
            __builtin_amdgcn_wave_barrier();
        }
        return;
    }
    // rolled: unrolled, the activation's code would not fit the instruction cache (8192 x 2048 x 8512 took 349 us, not 286)
    auto rows = [&](int i, auto whole) {
        constexpr bool kWhole = decltype(whole)::value;
#pragma unroll 1
        for (int p = 0; p < NP; ++p) {
            float v[4], bias[4], res[4];
            const int m = mw + i * 16 + row_of(p), n = nw + col_of(p);
            bias4(a, n, bias);
            res4<TO, kWhole>(a, m, n, res);
            staged(p, v);
            scale4_any<KIND>(a, m, n, v);
            finish4<TO, EPI, kWhole>(a, m, n, v, bias, res);
        }
    };
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        stage(i);
        if (a.whole) rows(i, std::true_type{});
        else rows(i, std::false_type{});
        __builtin_amdgcn_wave_barrier();
    }
}

// The splits' parts of y, added in order, and the epilogue. y, the residual,
// z and a part are each one run of M N values, of which a thread takes 4; a
// part's stride is a multiple of 4. INT: the parts are integers, whose sum the row's and the column's scale then
// multiply, and a name of its own in each of the two builds of this file.
template <bool INT, typename TO>
__global__ __launch_bounds__(256) void k_join(LinearArgs a) {
    const int64_t total = (int64_t)a.M * a.N, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= total) return;
    const int left = (int)min((int64_t)4, total - i);
    const float *p = a.part + i;
    float v[4] = {0.f, 0.f, 0.f, 0.f}, z[4], res[4];
    const int64_t step = part_stride(a.M, a.N);
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s, p += step) {
        const f32x4 c = *reinterpret_cast<const f32x4 *>(p);  // behind the last value: the stride's rest
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = INT ? add_bits(v[e], c[e]) : v[e] + c[e];
    }
    int64_t m = i / a.N;
    int n = (int)(i - m * a.N);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (INT && e < left) v[e] = scaled(v[e], a.xs[m], a.ws[n]);
        if (a.bias && e < left) v[e] += a.bias[n];
        if (++n == a.N) n = 0, ++m;
        z[e] = v[e];
    }
    if (a.pre) put4<TO>(reinterpret_cast<TO *>(a.pre) + i, z, left, left == 4);
    if (a.res) {
        get4<TO>(res, reinterpret_cast<const TO *>(a.res) + i, left, left == 4);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) res[e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (a.act == SSD_ACT_SILU) v[e] = act_of<sizeof(TO) == 2>(v[e], SSD_ACT_SILU);
        else if (a.act == SSD_ACT_GELU) v[e] = act_of<sizeof(TO) == 2>(v[e], SSD_ACT_GELU);
        v[e] += res[e];
    }
    put4<TO>(reinterpret_cast<TO *>(a.y) + i, v, left, left == 4);
}

// 16 bytes from a multiple of B bytes. A load of 16 bytes from an odd multiple of 2 takes twice the
// time of one from a multiple of 4: there the 5 words around them are loaded, and shifted. (The
// fifth is read 2 bytes further than the 16; the callers' rows go on for at least that much.)
template <int B>
__device__ __forceinline__ u32x4 ld_any(const char *p) {
    typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(4)));
    if constexpr (B == 4) return *reinterpret_cast<const u32x4_any *>(p);
    const uint32_t by = (uint32_t)(uintptr_t)p & 2u;
    const u32x4 q = *reinterpret_cast<const u32x4_any *>(p - by);
    const uint32_t last = *reinterpret_cast<const uint32_t *>(p + 12 + by);  // by = 0: of the 16 themselves
    return u32x4{__builtin_amdgcn_alignbyte(q[1], q[0], by), __builtin_amdgcn_alignbyte(q[2], q[1], by),
                 __builtin_amdgcn_alignbyte(q[3], q[2], by), __builtin_amdgcn_alignbyte(last, q[3], by)};
}
// B: the bytes that every row begins at a multiple of. 16: loads through resources that end with
// the operand; 4 and 2: whole steps by address and the last one value by value
// (13 x 7469 x 3392 in bf16: 21 us, 38 with copies in rows of 16-byte multiples in front).
// C: blocks of 16 rows of w that a work-group takes.
template <int KIND, typename TO, int B, int C>
__global__ __launch_bounds__(512) void k_skinny(LinearArgs a) {
    __shared__ __attribute__((aligned(16))) float red[8][64][4];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int r = lane & 15, kg = lane >> 4;
    const int n0 = blockIdx.x * (16 * C);
    const int cols = min(16 * C, a.N - n0);
    f32x4 acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
    // U steps' operands are loaded before the first is used; steps behind the last are zeros
    constexpr int U = C == 1 ? 4 : 2;
    if constexpr (B < 16) {
        // rows behind the last take the last one's place: their results are not stored
        const char *xr = reinterpret_cast<const char *>(a.x) + (int64_t)min(r, a.M - 1) * a.ldx;
        const char *wr[C];
#pragma unroll
        for (int c = 0; c < C; ++c) wr[c] = reinterpret_cast<const char *>(a.w) + (int64_t)min(n0 + c * 16 + r, a.N - 1) * a.ldw;
        const int whole = (int)(a.kbytes / 128u);
        for (int s0 = w; s0 < whole; s0 += 8 * U) {
            u32x4 wl[U][C], wh[U][C], xl[U], xh[U];
            uint32_t keep[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool live = s0 + 8 * u < whole;
                const uint32_t c0 = (uint32_t)(live ? s0 + 8 * u : 0) * 128u + kg * 16u;
                keep[u] = live ? ~0u : 0u;
#pragma unroll
                for (int c = 0; c < C; ++c) wl[u][c] = ld_any<B>(wr[c] + c0), wh[u][c] = ld_any<B>(wr[c] + c0 + 64);
                xl[u] = ld_any<B>(xr + c0);
                xh[u] = ld_any<B>(xr + c0 + 64);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int c = 0; c < C; ++c)
                    acc[c] = mma2<KIND>(wl[u][c] & keep[u], wh[u][c] & keep[u], xl[u] & keep[u], xh[u] & keep[u], acc[c], 0, 0);
        }
        if (whole < a.steps && w == whole % 8) {  // the step that the rows end in
            const uint32_t c0 = (uint32_t)whole * 128u + kg * 16u, c1 = c0 + 64u;
            const u32x4 xl = ld_rest<TO>(xr, c0, a.kbytes), xh = ld_rest<TO>(xr, c1, a.kbytes);
#pragma unroll
            for (int c = 0; c < C; ++c)
                acc[c] = mma2<KIND>(ld_rest<TO>(wr[c], c0, a.kbytes), ld_rest<TO>(wr[c], c1, a.kbytes), xl, xh, acc[c], 0, 0);
        }
    } else {
        const rsrc_t rw = make_rsrc(reinterpret_cast<const char *>(a.w) + (int64_t)n0 * a.ldw, (uint32_t)(cols * a.ldw));
        const rsrc_t rx = make_rsrc(a.x, (uint32_t)(a.M * a.ldx));
        rsrc_t rsw = rw, rsx = rx;
        if constexpr (KIND == kMX) {
            rsw = make_rsrc(a.wscale + (int64_t)n0 * a.lds, (uint32_t)(cols * a.lds));
            rsx = make_rsrc(a.xscale, (uint32_t)(a.M * a.lds));
        }
        const uint32_t ldx = (uint32_t)a.ldx, ldw = (uint32_t)a.ldw, ldsc = (uint32_t)a.lds;
        for (int s0 = w; s0 < a.steps; s0 += 8 * U) {
            u32x4 wl[U][C], wh[U][C], xl[U], xh[U];
            int sw[U][C], sx[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t c0 = (uint32_t)(s0 + 8 * u) * 128u + kg * 16u, c1 = c0 + 64u;
                const uint32_t o0 = oob_if(c0 >= a.kbytes, c0), o1 = oob_if(c1 >= a.kbytes, c1);
                const uint32_t b = (uint32_t)(s0 + 8 * u) * 4u + kg, ob = oob_if(b >= ldsc, b);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const uint32_t row = c * 16 + r;
                    wl[u][c] = buf_ld128(rw, o0 + row * ldw);
                    wh[u][c] = buf_ld128(rw, o1 + row * ldw);
                    sw[u][c] = KIND == kMX ? (int)__builtin_amdgcn_raw_buffer_load_b8(rsw, ob + row * ldsc, 0, 0) : 0;
                }
                xl[u] = buf_ld128(rx, o0 + r * ldx);
                xh[u] = buf_ld128(rx, o1 + r * ldx);
                sx[u] = KIND == kMX ? (int)__builtin_amdgcn_raw_buffer_load_b8(rsx, ob + r * ldsc, 0, 0) : 0;
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int c = 0; c < C; ++c) acc[c] = mma2<KIND>(wl[u][c], wh[u][c], xl[u], xh[u], acc[c], sw[u][c], sx[u]);
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (c) __syncthreads();
        *reinterpret_cast<f32x4 *>(red[w][lane]) = acc[c];
        __syncthreads();
        if (w == c) {
            float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const f32x4 q = *reinterpret_cast<const f32x4 *>(red[k][lane]);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = KIND == kInt ? add_bits(v[e], q[e]) : v[e] + q[e];
            }
            scale4_any<KIND>(a, r, n0 + c * 16 + kg * 4, v);
            finish4_any<TO>(a, r, n0 + c * 16 + kg * 4, v);
        }
    }
}

// The rows of two operands (R1 of in1, R2 of in2, n values each) copied to rows
// of ldo values (whole multiples of 16 bytes), zeros behind them: for operands whose
// rows k_tile's loads cannot take. A wavefront takes 64 groups of 16 bytes of a row.
template <typename U>
__global__ __launch_bounds__(256) void k_pad(const U *in1, U *out1, int64_t R1, const U *in2, U *out2, int64_t R2, int n,
                                             int ldo) {
    constexpr int E = 16 / sizeof(U);
    int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int c = ((int)blockIdx.y * 64 + (threadIdx.x & 63)) * E;
    if (row >= R1 + R2 || c >= ldo) return;
    const bool first = row < R1;
    if (!first) row -= R1;
    const U *p = (first ? in1 : in2) + row * n + c;
    union {
        U u[E];
        u32x4 v;
    } q;
#pragma unroll
    for (int e = 0; e < E; ++e) q.u[e] = c + e < n ? p[e] : (U)0;
    U *o = (first ? out1 : out2) + row * ldo + c;
    if (sizeof(U) > 1) {
        *reinterpret_cast<u32x4 *>(o) = q.v;
    } else {  // scales: rows of multiples of 4
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (c + e < ldo) o[e] = q.u[e];
    }
}

// out (C x ldo) = in (R x C) transposed, zeros behind column R. 64 x 64 a work-group.
// fp32's gradients take it. With many rows its products are bound by the matrix cores, beside which these
// copies are small; with few, they are most of the call (3 x 4800 x 11144: w's alone 107 us of 268, where a library
// product takes 135 for both gradients).
template <typename T>
__global__ __launch_bounds__(256) void k_transpose(const T *in, T *out, int R, int C, int ldo) {
    __shared__ T sm[64][64 + 4 / sizeof(T)];
    const int r0 = blockIdx.x * 64, c0 = blockIdx.y * 64, x = threadIdx.x & 63, y = threadIdx.x >> 6;
    for (int i = y; i < 64; i += 4)
        sm[i][x] = (r0 + i < R && c0 + x < C) ? in[(int64_t)(r0 + i) * C + c0 + x] : (T)0.f;
    __syncthreads();
    for (int i = y; i < 64; i += 4)
        if (c0 + i < C && r0 + x < ldo) out[(int64_t)(c0 + i) * ldo + r0 + x] = sm[x][i];
}

// dz = dy act'(z), rows of ldz values with zeros behind column N, and the
// shares of db of each R rows (fp32, before dz is rounded). In bf16 dz is rounded to it, as an operand of the
// matrix cores' products has to be (two parts of it would double both products): the gradients are then off by
// 2.3e-3 of their size on ordinary data, where rounding them alone makes 1.7e-3. A work-group
// takes R rows of 512 columns, a lane 8 columns (V: N is a multiple of 8 and
// they are one load) of every Y-th row. Bound: HBM, two reads and one
// write (16384 x 3352 in bf16, SiLU: 330 MB in 67 us, 4.9 TB/s, what a copy reaches).
// Y wavefronts: 4, or 16 where there are fewer than 4 work-groups for a CU and the time is
// the chain of a wavefront's rows (7676 x 108 in bf16 9.1 us, with 4 of 64 rows 29.9; 933 x 430 7.8 and 25.8).
template <typename T, bool V, int ACT, int Y>
__global__ __launch_bounds__(64 * Y) void k_dz(const T *dy, const T *pre, T *dz, float *part, int M, int N, int ldz, int R) {
    __shared__ float col[Y][64][8];
    const int lane = threadIdx.x & 63, y = threadIdx.x >> 6;
    const int m0 = blockIdx.x * R, n = blockIdx.y * 512 + lane * 8;
    float sum[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = 0.f;
#pragma unroll 4
    for (int i = y; i < R; i += Y) {
        const int m = m0 + i;
        if (m >= M || n >= ldz) continue;
        const int64_t at = (int64_t)m * N + n;
        float v[8], z[8];
        if (V && n >= N) {  // between the row's end and ldz
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = z[e] = 0.f;
        } else if constexpr (V) {
            float lo[4], hi[4];
            get4<T>(lo, dy + at, 4, true);
            get4<T>(hi, dy + at + 4, 4, true);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = lo[e], v[4 + e] = hi[e];
            if constexpr (ACT != SSD_ACT_NONE) {
                get4<T>(lo, pre + at, 4, true);
                get4<T>(hi, pre + at + 4, 4, true);
#pragma unroll
                for (int e = 0; e < 4; ++e) z[e] = lo[e], z[4 + e] = hi[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = n + e < N ? (float)dy[at + e] : 0.f;
                z[e] = (ACT != SSD_ACT_NONE && n + e < N) ? (float)pre[at + e] : 0.f;
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (ACT != SSD_ACT_NONE) v[e] *= act_slope<sizeof(T) == 2>(z[e], ACT);
            sum[e] += v[e];
        }
        if (dz) {
            const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
            T *o = dz + (int64_t)m * ldz + n;  // ldz is a multiple of 16 bytes
            put4<T>(o, lo, 4, true);
            if (n + 4 < ldz) put4<T>(o + 4, hi, 4, true);
        }
    }
    if (!part) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) col[y][lane][e] = sum[e];
    __syncthreads();
    if (y == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
            for (int k = 1; k < Y; ++k) sum[e] += col[k][lane][e];
            if (n + e < N) part[(int64_t)blockIdx.x * N + n + e] = sum[e];
        }
    }
}

// How a product is formed. bm = 0: k_skinny, else a work-group's tile of y.
// The model of a tile kernel's time, in microseconds: work-groups run in rounds over
// the 256 CUs (2 of the 128-tiles, 4 of the 64-tiles share a CU), each round
// its steps of 128 bytes along k and a fixed share for the start and the
// epilogue; a split of the sum over k adds a launch and the traffic of its fp32
// parts. A step's time is measured (large products on a warm GPU): of the bf16 and
// 8-bit tiles the matrix cores' for the largest one, more and more LDS's and
// the loads' for the smaller ones; of fp32 the matrix cores' for each, or the
// vector unit's, which splits the operands. A last round that leaves CUs fewer work-groups has shorter steps,
// down to `least` of them. Of 40 products of 32 to 8192 rows the plan so chosen takes 1.6% (bf16)
// and 2.4% (fp32) more than the best one on average, with full last rounds 4.7% and 8.9%
// (777 x 1003 x 515 in fp32: 18 us in 4 parts, 22 in 8).
#ifndef SSD_INT_TU
LinearPlan linear_plan(int64_t M, int64_t N, int64_t kbytes, bool f32, bool along_k) {
    LinearPlan p = {};
    p.steps = (int)((kbytes + 127) / 128);
    p.splits = 1;
    p.steps_per_split = p.steps;
    if (M <= 16 && !along_k) return p;
    struct Tile {
        int bm, bn;
        int64_t slots;
        double step, step32, fixed, least, least32;
    };
    const Tile tiles[] = {{256, 256, 256, 1.45, 0, 14, 1, 1}, {256, 192, 256, 1.22, 3.3, 12, 1, 1},
                          {128, 128, 512, 0.9, 2.3, 8, 1, 0.8}, {64, 64, 1024, 0.6, 1.5, 5, 0.6, 0.35}};
    // the time of n columns by one tile's kernel, and its plan
    auto plan_of = [&](const Tile &c, int64_t n, int splits, LinearPlan *q) {
        const int per = ((p.steps + splits - 1) / splits + 1) & ~1;  // steps go in pairs
        if (splits > 1 && (p.steps + per - 1) / per != splits) return 1e300;
        const int64_t nm = (M + c.bm - 1) / c.bm, nn = (n + c.bn - 1) / c.bn;
        const int64_t work = nm * nn * splits, full = work / c.slots, last = work % c.slots;
        *q = p;
        q->bm = c.bm;
        q->bn = c.bn;
        q->splits = splits;
        q->steps_per_split = per;
        q->nm = (int)nm;
        q->nn = (int)nn;
        // operands along k: the small tiles' steps are slower (3352 x 16384 x 768: 128-tiles 118 us, 256-tiles 110)
        const double slow = along_k && c.bm < 256 ? 1.15 : 1.0;
        const double step = per * (f32 ? c.step32 : c.step) * slow, share = (double)last / c.slots,
                     least = f32 ? c.least32 : c.least;
        double t = full * (step + c.fixed);
        if (last) t += step * (share > least ? share : least) + c.fixed;
        if (splits > 1) t += 5 + 1.4 * splits * M * n * 4 / 5.0e6;
        return t;
    };
    double best = 1e300;
    LinearPlan q, top = p;
    auto best_of = [&](int64_t n, int most_splits, LinearPlan *out) {
        double t = 1e300;
        for (const Tile &c : tiles) {
            if (f32 && c.bn == 256) continue;  // its operands in three parts do not fit the registers
            for (int splits = 1; splits <= most_splits && splits <= p.steps; splits += splits < 8 ? 1 : 4) {
                const double u = plan_of(c, n, splits, &q);
                if (u < t) t = u, *out = q;
            }
        }
        return t;
    };
    best = best_of(N, 32, &top);
    // whole rounds of the large tile, and the columns that are left by the tile that is best for them
    // (8192 x 2048 x 8512 in 8 bits: 4 rounds and 320 columns, 176 us; 5 rounds, the last a quarter full, 194)
    if (!along_k) {
        const Tile &c = tiles[f32 ? 1 : 0];
        const int64_t nm = (M + c.bm - 1) / c.bm;
        int64_t nf = N / c.bn;
        while (nf > 0 && nm * nf % 256 != 0) --nf;
        LinearPlan rest;
        if (nf > 0 && nf * c.bn < N) {
            const double t = plan_of(c, nf * c.bn, 1, &q);
            const LinearPlan main = q;
            if (t + best_of(N - nf * c.bn, 1, &rest) < best) {
                top = main;
                top.n_main = (int)(nf * c.bn);
                top.rest_bm = rest.bm;
                top.rest_bn = rest.bn;
                top.rest_nm = rest.nm;
                top.rest_nn = rest.nn;
            }
        }
    }
    return top;
}
#endif  // SSD_INT_TU

template <int KIND, typename TO, bool XT, bool WT, bool RAGGED>
static ssd_status run_tile(const LinearArgs &a, const LinearPlan &p, hipStream_t s) {
    const dim3 grid((unsigned)(p.nm * p.nn), (unsigned)p.splits);
    auto go = [&](auto epi) {
        constexpr int EPI = decltype(epi)::value;
        if (p.bm == 64) return launch(k_tile<KIND, TO, 64, 64, 2, 2, EPI, XT, WT, RAGGED>, grid, dim3(256), s, a);
        if (p.bm == 128) return launch(k_tile<KIND, TO, 128, 128, 2, 2, EPI, XT, WT, RAGGED>, grid, dim3(256), s, a);
        if (p.bn == 192) return launch(k_tile<KIND, TO, 256, 192, 2, 4, EPI, XT, WT, RAGGED>, grid, dim3(512), s, a);
        if constexpr (KIND != kF32) return launch(k_tile<KIND, TO, 256, 256, 2, 4, EPI, XT, WT, RAGGED>, grid, dim3(512), s, a);
        return hipErrorInvalidValue;  // no such plan
    };
    hipError_t e;
    if (p.splits > 1) {
        e = go(std::integral_constant<int, kParts>{});
    } else if constexpr (XT || WT) {  // gradients have no activation
        e = go(std::integral_constant<int, SSD_ACT_NONE>{});
    } else {
        e = a.act == SSD_ACT_SILU   ? go(std::integral_constant<int, SSD_ACT_SILU>{})
            : a.act == SSD_ACT_GELU ? go(std::integral_constant<int, SSD_ACT_GELU>{})
                                    : go(std::integral_constant<int, SSD_ACT_NONE>{});
    }
    if (e == hipSuccess && p.splits > 1) {
        const int64_t n = ((int64_t)a.M * a.N + 3) / 4;
        e = launch(k_join<KIND == kInt, TO>, dim3((unsigned)((n + 255) / 256)), dim3(256), s, a);
    }
    return e == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

template <int KIND, typename TO>
static ssd_status run_linear(const LinearArgs &a, const LinearPlan &p, hipStream_t s) {
    if constexpr (KIND == kBF16 || KIND == kF32) {
        if (p.bm && a.kbytes % 16 != 0) return run_tile<KIND, TO, false, false, true>(a, p, s);
    }
    if (p.bm) return run_tile<KIND, TO, false, false, false>(a, p, s);
    auto go = [&](auto k, int columns) {
        return launch(k, dim3((unsigned)((a.N + columns - 1) / columns)), dim3(512), s, a) == hipSuccess ? SSD_OK : SSD_ERR_HIP;
    };
    auto of = [&](auto b) {
        constexpr int B = decltype(b)::value;
        // short rows are few steps a wavefront, beside which its start and the reads of x count: with many of
        // them a work-group takes 32 (8 x 768 x 50257 in bf16 23.8 us -> 17.1, 8 x 1024 x 32768 17.4 -> 12.8;
        // longer ones lose by it: 8 x 2048 x 50257 45.9 -> 51.1)
        return a.N >= 16384 && a.steps <= 24 ? go(k_skinny<KIND, TO, B, 2>, 32) : go(k_skinny<KIND, TO, B, 1>, 16);
    };
    if constexpr (KIND == kBF16) {
        if (a.kbytes % 4 != 0) return of(std::integral_constant<int, 2>{});
    }
    if constexpr (KIND == kBF16 || KIND == kF32) {
        if (a.kbytes % 16 != 0) return of(std::integral_constant<int, 4>{});
    }
    return of(std::integral_constant<int, 16>{});
}

// The plan's one product, or its two (n_main): one(args, plan) launches each.
template <typename F>
static ssd_status in_parts(LinearArgs a, const LinearPlan &p, int64_t es, F one) {
    auto go = [&](LinearArgs b, const LinearPlan &q) {
        b.nm = q.nm; b.nn = q.nn; b.steps = q.steps; b.splits = q.splits; b.steps_per_split = q.steps_per_split;
        if (q.splits == 1) b.part = nullptr;
        b.whole = (b.N & 3) == 0 && (b.ldy & 3) == 0;
        return one(b, q);
    };
    if (a.ldy == 0) a.ldy = a.N;
    if (!p.n_main) return go(a, p);
    // never with an operand along k
    const int64_t n = p.n_main;
    LinearArgs b = a;
    LinearPlan rest = p;
    rest.bm = p.rest_bm; rest.bn = p.rest_bn; rest.nm = p.rest_nm; rest.nn = p.rest_nn;
    a.N = (int)n;
    b.N -= (int)n;
    b.w = static_cast<const char *>(b.w) + n * b.ldw;
    if (b.wscale) b.wscale += n * b.lds;
    if (b.ws) b.ws += n;
    if (b.bias) b.bias += n;
    if (b.res) b.res = static_cast<const char *>(b.res) + n * es;
    if (b.pre) b.pre = static_cast<char *>(b.pre) + n * es;
    b.y = static_cast<char *>(b.y) + n * es;
    const ssd_status st = go(a, p);
    return st != SSD_OK ? st : go(b, rest);
}

#ifdef SSD_INT_TU
ssd_status launch_linear_int(const LinearArgs &a, const LinearPlan &p, ssd_dtype dtype, hipStream_t s) {
    return in_parts(a, p, dtype == SSD_BF16 ? 2 : 4, [&](const LinearArgs &b, const LinearPlan &q) {
        return dtype == SSD_BF16 ? run_linear<kInt, bf16>(b, q, s) : run_linear<kInt, float>(b, q, s);
    });
}
#else
ssd_status launch_linear(LinearArgs a, const LinearPlan &p, bool mx, ssd_dtype dtype, hipStream_t s) {
    return in_parts(a, p, dtype == SSD_BF16 ? 2 : 4, [&](const LinearArgs &b, const LinearPlan &q) {
        if (mx) return run_linear<kMX, bf16>(b, q, s);
        if (b.wt) return b.xt ? run_tile<kBF16, bf16, true, true, false>(b, q, s) : run_tile<kBF16, bf16, false, true, false>(b, q, s);
        return dtype == SSD_BF16 ? run_linear<kBF16, bf16>(b, q, s) : run_linear<kF32, float>(b, q, s);
    });
}

template <typename U>
static ssd_status run_pad(const void *in1, void *out1, int64_t R1, const void *in2, void *out2, int64_t R2, int64_t n,
                          int64_t ldo, hipStream_t s) {
    return launch(k_pad<U>, dim3((unsigned)((R1 + R2 + 3) / 4), (unsigned)((ldo * sizeof(U) + 1023) / 1024)), dim3(256), s, (const U *)in1, (U *)out1, R1,
                  (const U *)in2, (U *)out2, R2, (int)n, (int)ldo) == hipSuccess
               ? SSD_OK
               : SSD_ERR_HIP;
}
ssd_status launch_pad(const void *in1, void *out1, int64_t R1, const void *in2, void *out2, int64_t R2, int64_t n,
                      int64_t ldo, int es, hipStream_t s) {
    if (es == 1) return run_pad<uint8_t>(in1, out1, R1, in2, out2, R2, n, ldo, s);
    if (es == 2) return run_pad<uint16_t>(in1, out1, R1, in2, out2, R2, n, ldo, s);
    return run_pad<uint32_t>(in1, out1, R1, in2, out2, R2, n, ldo, s);
}

ssd_status launch_transpose(const void *in, void *out, int64_t R, int64_t C, int64_t ldo, hipStream_t s) {
    const dim3 grid((unsigned)((ldo + 63) / 64), (unsigned)((C + 63) / 64)), block(256);
    return launch(k_transpose<float>, grid, block, s, (const float *)in, (float *)out, (int)R, (int)C, (int)ldo) ==
                   hipSuccess
               ? SSD_OK
               : SSD_ERR_HIP;
}

// Rows of a share of db: 64, or 16 where those were fewer work-groups than CUs.
int dz_rows(int64_t M, int64_t ldz) { return (M + 63) / 64 * ((ldz + 511) / 512) < 256 ? 16 : 64; }

template <typename T>
static ssd_status run_dz(const void *dy, const void *pre, int act, void *dz, float *part, int64_t M, int64_t N, int64_t ldz,
                         hipStream_t s) {
    const int R = dz_rows(M, ldz);
    const dim3 grid((unsigned)((M + R - 1) / R), (unsigned)((ldz + 511) / 512));
    const bool few = (int64_t)grid.x * grid.y < 1024;
    auto go = [&](auto k) {
        return launch(k, grid, dim3(few ? 1024 : 256), s, (const T *)dy, (const T *)pre, (T *)dz, part, (int)M, (int)N, (int)ldz,
                      R) == hipSuccess
                   ? SSD_OK
                   : SSD_ERR_HIP;
    };
    auto by_act = [&](auto v) {
        constexpr bool V = decltype(v)::value;
        if (act == SSD_ACT_SILU) return few ? go(k_dz<T, V, SSD_ACT_SILU, 16>) : go(k_dz<T, V, SSD_ACT_SILU, 4>);
        if (act == SSD_ACT_GELU) return few ? go(k_dz<T, V, SSD_ACT_GELU, 16>) : go(k_dz<T, V, SSD_ACT_GELU, 4>);
        return few ? go(k_dz<T, V, SSD_ACT_NONE, 16>) : go(k_dz<T, V, SSD_ACT_NONE, 4>);
    };
    return N % 8 == 0 ? by_act(std::true_type{}) : by_act(std::false_type{});
}

ssd_status launch_dz(const void *dy, const void *pre, int act, void *dz, float *part, int64_t M, int64_t N, int64_t ldz,
                     ssd_dtype dtype, hipStream_t s) {
    return dtype == SSD_BF16 ? run_dz<bf16>(dy, pre, act, dz, part, M, N, ldz, s)
                             : run_dz<float>(dy, pre, act, dz, part, M, N, ldz, s);
}
#endif  // SSD_INT_TU

}  // namespace ssd
