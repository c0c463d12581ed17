// Beam search's choice of the next tokens for gfx950: over all beams k and
// vocabulary entries v of a sequence, the `beams` largest
//
//   cand[k, v] = score[k] + logits[k, v] - log sum_u exp(logits[k, u])
//
// in order, equal ones by the lowest k V + v. A finished beam has the one
// candidate (k, eos) at score[k]; whatever is not a number counts as -inf.
//
// Bound: HBM, one read of the logits. k_beam_top gives each wavefront 2048
// logits of a row, which stay in registers: it sums their exponentials and
// finds their `beams` largest. Within a row cand orders as the logits do, so
// that needs no sum. A filter leaves few to be sorted: the beams-th largest of
// the 64 lanes' own maxima is a lower bound on the beams-th largest value, and
// of 2048 values about 18 reach it at 16 beams. k_beam_pick (one work-group
// per sequence, a wavefront per beam) merges a row's lists the same way,
// forms the scores and merges the beams.
// 64 x 8 x 65536 fp32 logits: 134 MB in 30 us, 4.5 TB/s, and 10 us to pick; one
// sequence of 4 beams and 50257 bf16 logits: 7 and 6 us, latency.
//
// The sums of exponentials are fp32 within 2048 logits and 64-bit across them, and scores
// are compared in 64 bits, so that two candidates of different beams change places only where
// they are closer than the exponentials' own error: a term e^-d is off by under (d + 1) 2^-22 of
// itself (2^x in fp32 of a difference and a product rounded to it), the sum by less, since the
// errors differ in sign. (With a lane's sum in fp32 over 2^28 equal logits, it was 3e-5.)
#include <float.h>

#include "ssd_common.h"
#include "ssd_internal.h"

namespace ssd {

constexpr int kTile = 2048;        // logits a wavefront holds at a time, 32 a lane
constexpr int kPerLane = kTile / 64;

// Order-preserving bits of a float (no NaN): larger floats, larger bits; 0 is below all.
// Both zeros are one value (-0 + 0 = 0): they tie.
__device__ __forceinline__ uint32_t ord32(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);
    return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ord32(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o ^ 0x80000000u) : ~o);
}
constexpr uint32_t kNone = 0x007fffffu;  // ord32(-inf)
// Larger value first, then lower index: one 64-bit comparison. 0 is no entry.
__device__ __forceinline__ uint64_t key_of(uint32_t ord, uint32_t idx) { return ((uint64_t)ord << 32) | (uint32_t)~idx; }

// The value of lane ^ m, on the vector unit (a shuffle through LDS would take some 10
// times as long): within quads, halves and rows of 16 by DPP, across rows by
// swapping halves of two registers.
template <int m>
__device__ __forceinline__ uint32_t xor32(uint32_t v) {
    const int i = (int)v;
    if constexpr (m == 1) return (uint32_t)__builtin_amdgcn_mov_dpp(i, 0xb1, 0xf, 0xf, true);        // quad 1 0 3 2
    if constexpr (m == 2) return (uint32_t)__builtin_amdgcn_mov_dpp(i, 0x4e, 0xf, 0xf, true);        // quad 2 3 0 1
    if constexpr (m == 4) return xor32<1>(xor32<2>((uint32_t)__builtin_amdgcn_mov_dpp(i, 0x141, 0xf, 0xf, true)));  // 7 - l, then ^ 3
    if constexpr (m == 8) return (uint32_t)__builtin_amdgcn_mov_dpp(i, 0x128, 0xf, 0xf, true);       // rotated by 8
    if constexpr (m == 16) {
        const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return (threadIdx.x & 16) ? p[0] : p[1];
    }
    if constexpr (m == 32) {
        const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return (threadIdx.x & 32) ? p[0] : p[1];
    }
    return v;
}
template <int m>
__device__ __forceinline__ uint64_t xor64(uint64_t v) {
    return ((uint64_t)xor32<m>((uint32_t)(v >> 32)) << 32) | xor32<m>((uint32_t)v);
}
template <int m>
__device__ __forceinline__ float xorf(float v) { return __uint_as_float(xor32<m>(__float_as_uint(v))); }
template <int m>
__device__ __forceinline__ double xord(double v) { return __longlong_as_double((long long)xor64<m>((uint64_t)__double_as_longlong(v))); }

template <typename U, int j>
__device__ __forceinline__ U exchange(U v, int lane, bool up) {
    U o;
    if constexpr (sizeof(U) == 8) o = xor64<j>(v); else o = xor32<j>(v);
    const bool keep_max = up == ((lane & j) == 0);
    return (keep_max == (v > o)) ? v : o;
}
template <typename U, int j>
__device__ __forceinline__ U merge_steps(U v, int lane, bool up) {
    v = exchange<U, j>(v, lane, up);
    if constexpr (j > 1) v = merge_steps<U, j / 2>(v, lane, up);
    return v;
}
// Bitonic sort of one value per lane, largest in lane 0.
template <typename U>
__device__ __forceinline__ U sort_desc(U v, int lane) {
    v = merge_steps<U, 1>(v, lane, (lane & 2) == 0);
    v = merge_steps<U, 2>(v, lane, (lane & 4) == 0);
    v = merge_steps<U, 4>(v, lane, (lane & 8) == 0);
    v = merge_steps<U, 8>(v, lane, (lane & 16) == 0);
    v = merge_steps<U, 16>(v, lane, (lane & 32) == 0);
    return merge_steps<U, 32>(v, lane, true);
}

template <int m = 32>
__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
    const uint64_t o = xor64<m>(v);
    v = o > v ? o : v;
    if constexpr (m > 1) v = wave_max64<m / 2>(v);
    return v;
}
template <int m = 32>
__device__ __forceinline__ float wave_maxf(float v) {
    v = fmaxf(v, xorf<m>(v));
    if constexpr (m > 1) v = wave_maxf<m / 2>(v);
    return v;
}
template <int m = 32>
__device__ __forceinline__ float wave_sumf(float v) {
    v += xorf<m>(v);
    if constexpr (m > 1) v = wave_sumf<m / 2>(v);
    return v;
}
template <int m = 32>
__device__ __forceinline__ double wave_sumd(double v) {
    v += xord<m>(v);
    if constexpr (m > 1) v = wave_sumd<m / 2>(v);
    return v;
}

// e^d, d <= 0, to 1e-11: 2^n e^r with |r| <= ln 2 / 2 and the series up to r^9. For the rises of a list's largest
// logit, whose factors' errors multiply: fp32's would be up to 1e-4 after 2048 of them.
__device__ __forceinline__ double exp_neg(double d) {
    const double y = fmax(d * 1.4426950408889634, -1100.0), n = rint(y), r = (y - n) * 0.6931471805599453;
    double p = 1.0 / 362880;
    const double c[] = {1.0 / 40320, 1.0 / 5040, 1.0 / 720, 1.0 / 120, 1.0 / 24, 1.0 / 6, 0.5, 1.0, 1.0};
#pragma unroll
    for (int i = 0; i < 9; ++i) p = fma(p, r, c[i]);
    return ldexp(p, (int)n);
}

// The sorted list in lanes 0 .. K-1 and the n <= 64 - K keys in buf, merged.
__device__ __forceinline__ uint64_t merge_into(uint64_t best, const uint64_t *buf, int n, int K, int lane) {
    uint64_t v = lane < K ? best : 0;
    if (lane >= K && lane - K < n) v = buf[lane - K];
    return sort_desc(v, lane);
}

// At most 168 registers, as many as leave a SIMD three wavefronts: the compiler hoists exp_neg's constants out of the
// loop and takes 193 (64 x 8 x 65536 logits: 52.4 us in all).
template <typename T>
__global__ __launch_bounds__(256, 3) void k_beam_top(BeamArgs a) {
    constexpr int VE = 16 / (int)sizeof(T);    // logits per 16-byte load
    constexpr int NL = kPerLane / VE;          // loads per lane and tile
    __shared__ uint64_t bufs[4][64];
    const int lane = threadIdx.x & 63;
    uint64_t *buf = bufs[threadIdx.x >> 6];
    const int64_t gl = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t row = gl / a.lists;
    const int li = (int)(gl - row * a.lists);
    if (row >= a.rows || (a.finished && a.finished[row])) return;
    const int K = a.beams, V = a.V;
    const T *rp = reinterpret_cast<const T *>(a.logits) + row * V;
    uint64_t best = 0;
    float M = -INFINITY;
    double S = 0.0;
    for (int j = 0; j < a.tiles; ++j) {
        const int base = (li * a.tiles + j) * kTile;
        if (base >= V) break;
        float v[kPerLane];
        if (base + kTile <= V) {
            // a row of an odd number of logits begins at any multiple of its type. The split goes by
            // the place in the row all the same, so that equal rows have bit-equal sums (and tie)
            typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
            u32x4 raw[NL];
#pragma unroll
            for (int l = 0; l < NL; ++l) raw[l] = *reinterpret_cast<const u32x4_any *>(rp + base + (l * 64 + lane) * VE);
#pragma unroll
            for (int e = 0; e < kPerLane; ++e) {
                float f;
                if constexpr (sizeof(T) == 2) {
                    const uint32_t w = raw[e / VE][(e % VE) >> 1];
                    f = __uint_as_float((e & 1) ? (w & 0xffff0000u) : (w << 16));
                } else {
                    const uint32_t w = raw[e / VE][e % VE];
                    f = __uint_as_float(w);
                }
                v[e] = fmaxf(f, -INFINITY);  // NaN: -inf
            }
        } else {
#pragma unroll
            for (int e = 0; e < kPerLane; ++e) {
                const int i = base + ((e / VE) * 64 + lane) * VE + e % VE;
                const float f = i < V ? (float)rp[i] : -INFINITY;
                v[e] = fmaxf(f, -INFINITY);  // NaN: -inf
            }
        }
        float lm = v[0];
#pragma unroll
        for (int e = 1; e < kPerLane; ++e) lm = fmaxf(lm, v[e]);
        // these logits' sum, relative to the largest so far
        const float Mn = fmaxf(M, wave_maxf(lm));
        float s = 0.f;
        if (Mn > -INFINITY) {
#pragma unroll
            for (int e = 0; e < kPerLane; ++e) s += fast_exp2((v[e] - Mn) * kLog2e);
            s = wave_sumf(s);
        }
        // lower bound on the K-th largest of the tile and of the list so far; -inf is no candidate
        uint32_t bound = (uint32_t)__builtin_amdgcn_readlane((int)sort_desc(ord32(lm), lane), K - 1);
        const uint32_t kth = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(best >> 32), K - 1);
        bound = bound > kth ? bound : kth;
        const float least = bound > kNone ? from_ord32(bound) : -FLT_MAX;
        int n = 0;
#pragma unroll
        for (int e = 0; e < kPerLane; ++e) {
            const uint64_t mask = __ballot(v[e] >= least);  // (places behind the row hold -inf)
            if (mask) {
                const int i = base + ((e / VE) * 64 + lane) * VE + e % VE;
                const int at = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
                if (v[e] >= least && at < 64 - K) buf[at] = key_of(ord32(v[e]), (uint32_t)i);
                n += __popcll(mask);
            }
        }
        if (n <= 64 - K) {
            __builtin_amdgcn_wave_barrier();
            best = merge_into(best, buf, n, K, lane);
            __builtin_amdgcn_wave_barrier();
        } else {
            // many equal or ordered logits: the K largest one by one
            uint64_t fresh = 0, last = ~0ull;
            for (int k = 0; k < K; ++k) {
                uint64_t top = 0;
#pragma unroll
                for (int e = 0; e < kPerLane; ++e) {
                    const int i = base + ((e / VE) * 64 + lane) * VE + e % VE;
                    const uint64_t q = (i < V) ? key_of(ord32(v[e]), (uint32_t)i) : 0;
                    if (q < last && q > top) top = q;
                }
                last = wave_max64(top);
                if (lane == k) fresh = last;
                if (last == 0) break;
            }
            if (lane < K) buf[lane] = fresh;
            __builtin_amdgcn_wave_barrier();
            best = merge_into(best, buf, K, K, lane);
            __builtin_amdgcn_wave_barrier();
        }
        // the list's, in 64 bits (here, where the logits' registers are free)
        if (Mn > M) {
            if (M > -INFINITY) S *= exp_neg((double)M - (double)Mn);
            M = Mn;
        }
        S += (double)s;
    }
    if (lane < K) a.keys[gl * K + lane] = best;
    if (lane == 0) a.sums[gl] = S;  // relative to the first key's logit
}

// The larger score (equal ones: the lower lane) of 16 lanes; 0xffff: none.
template <int m>
__device__ __forceinline__ void better(double &s, uint32_t &who) {
    const double os = xord<m>(s);
    const uint32_t ow = xor32<m>(who);
    const bool take = ow != 0xffffu && (who == 0xffffu || os > s || (os == s && ow < who));
    s = take ? os : s;
    who = take ? ow : who;
    if constexpr (m > 1) better<m / 2>(s, who);
}

template <typename T>
__global__ __launch_bounds__(1024) void k_beam_pick(BeamArgs a) {
    constexpr int kMost = 16;  // beams
    __shared__ uint64_t bufs[kMost][64];
    __shared__ double sc[kMost][kMost];
    __shared__ uint32_t ix[kMost][kMost];
    __shared__ int cnt[kMost];
    __shared__ int live[kMost];   // 1: the row's candidates are its logits; 2: finished; 0: none
    const int lane = threadIdx.x & 63, k = threadIdx.x >> 6;
    const int K = a.beams, V = a.V;
    const int64_t b = blockIdx.x, row = b * K + k;
    // everything the row needs, loaded at once (what k_beam_top left of a finished row is not used)
    const bool in = lane < a.lists;
    const int64_t list = row * a.lists + (in ? lane : 0);
    const double sum = in ? a.sums[list] : 0.0;
    uint64_t key[kMost];
#pragma unroll
    for (int r = 0; r < kMost; ++r) key[r] = (in && r < K) ? a.keys[list * K + r] : 0;
    const float score = a.scores[row];
    const bool alive = score > -INFINITY;  // false for NaN too
    if (a.finished && a.finished[row]) {
        if (lane == 0) {
            live[k] = 2;
            cnt[k] = alive ? 1 : 0;
            sc[k][0] = (double)score;
            ix[k][0] = (uint32_t)a.eos;
        }
    } else {
        // log-sum-exp of the row
        const float top = key[0] ? from_ord32((uint32_t)(key[0] >> 32)) : -INFINITY;
        const float M = wave_maxf(top);
        const double S = wave_sumd(top > -INFINITY ? sum * exp((double)top - (double)M) : 0.0);
        const double lse = (double)M + log(S);
        const bool ok = alive && lse - lse == 0.0;  // a finite sum
        uint64_t best = 0;
        if (ok) {
            const uint64_t heads = sort_desc(key[0], lane);
            const uint64_t bound = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(heads >> 32), K - 1) << 32) |
                                   (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)heads, K - 1);
            int n = 0;
#pragma unroll
            for (int r = 0; r < kMost; ++r) {
                // keys differ, so at most K - 1 lists and the bound's own reach it
                const bool hit = key[r] && key[r] >= bound;
                const uint64_t mask = __ballot(hit);
                const int c = __popcll(mask);
                if (c) {
                    if (n + c > 64 - K) {
                        __builtin_amdgcn_wave_barrier();
                        best = merge_into(best, bufs[k], n, K, lane);
                        __builtin_amdgcn_wave_barrier();
                        n = 0;
                    }
                    const int at = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
                    if (hit) bufs[k][at] = key[r];
                    n += c;
                }
            }
            __builtin_amdgcn_wave_barrier();
            best = merge_into(best, bufs[k], n, K, lane);
        }
        const float l = from_ord32((uint32_t)(best >> 32));
        const bool use = ok && lane < K && best && l > -INFINITY;
        if (use) {
            sc[k][lane] = (double)score + ((double)l - lse);
            ix[k][lane] = (uint32_t)~(uint32_t)best;
        }
        const uint64_t used = __ballot(use);  // a leading run of lanes: the list is sorted
        if (lane == 0) {
            cnt[k] = __popcll(used);
            live[k] = ok ? 1 : 0;
        }
    }
    __syncthreads();
    if (k != 0) return;
    // the beams' lists, merged: lane j holds the head of beam j's
    int at = 0, got = 0;
    double hs = -INFINITY;
    uint32_t hi = 0xffffffffu;  // k V + v; beams in order, so equal scores go to the lower lane's
    const int mine = lane < K ? cnt[lane] : 0;
    if (mine > 0) hs = sc[lane][0], hi = ix[lane][0];
    for (; got < K; ++got) {
        double s = hs;
        uint32_t who = (mine > at) ? (uint32_t)lane : 0xffffu;
        better<8>(s, who);
        who = (uint32_t)__builtin_amdgcn_readfirstlane((int)who);
        if (who == 0xffffu) break;
        if (lane == (int)who) {
            const int64_t o = b * K + got;
            a.out_scores[o] = (float)hs;
            a.parent[o] = (int)(b * K + lane);
            a.token[o] = (int)hi;
            if (a.out_finished)
                a.out_finished[o] = ((a.finished && a.finished[b * K + lane]) || (int)hi == a.eos) ? 1 : 0;
            ++at;
            if (at < mine) hs = sc[lane][at], hi = ix[lane][at];
        }
    }
    // fewer candidates than beams: the lowest of those at -inf. Fewer than K
    // are not, so the first 2 K positions hold enough.
    for (int64_t i0 = 0; got < K && i0 < (int64_t)K * V; i0 += 64) {
        const int64_t i = i0 + lane;
        bool none = false;
        if (i < (int64_t)K * V) {
            const int kk = (int)(i / V), v = (int)(i - (int64_t)kk * V);
            if (cnt[kk] == 0) none = true;
            else if (live[kk] == 2) none = v != a.eos;
            else {
                const float f = (float)reinterpret_cast<const T *>(a.logits)[(b * K + kk) * V + v];
                none = !(f > -INFINITY);
            }
        }
        const uint64_t mask = __ballot(none);
        const int o = got + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
        if (none && o < K) {
            const int kk = (int)(i / V), v = (int)(i - (int64_t)kk * V);
            a.out_scores[b * K + o] = -INFINITY;
            a.parent[b * K + o] = (int)(b * K + kk);
            a.token[b * K + o] = v;
            if (a.out_finished)
                a.out_finished[b * K + o] = ((a.finished && a.finished[b * K + kk]) || v == a.eos) ? 1 : 0;
        }
        got += __popcll(mask);
    }
}

// Lists per row (at most 64, the lanes that merge them) and tiles per list.
void beam_plan(int64_t V, int *lists, int *tiles) {
    const int64_t t = (V + kTile - 1) / kTile;
    *tiles = (int)((t + 63) / 64);
    *lists = (int)((t + *tiles - 1) / *tiles);
}

template <typename T>
static ssd_status run_beam(const BeamArgs &a, int64_t batch, hipStream_t s) {
    const int64_t waves = a.rows * a.lists;
    if (launch(k_beam_top<T>, dim3((unsigned)((waves + 3) / 4)), dim3(256), s, a) != hipSuccess) return SSD_ERR_HIP;
    return launch(k_beam_pick<T>, dim3((unsigned)batch), dim3((unsigned)(64 * a.beams)), s, a) == hipSuccess
               ? SSD_OK
               : SSD_ERR_HIP;
}

ssd_status launch_beam_select(const BeamArgs &a, int64_t batch, ssd_dtype dtype, hipStream_t s) {
    return dtype == SSD_BF16 ? run_beam<bf16>(a, batch, s) : run_beam<float>(a, batch, s);
}

}  // namespace ssd
