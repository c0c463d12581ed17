// Embedding lookup for gfx950, y[r, :] = scale table[token[r], :], and the
// gradient of the table from its tokens in order:
//
//   dtable[v, :] = scale sum over r with token[r] = v of dy[r, :]
//
// in a fixed order, r ascending, so that the same inputs give the same bits. A
// token outside the table is a row of zeros, and adds to no gradient.
//
// k_sort: a work-group sorts up to 4096 tokens in LDS (stable, by digits of at
// most 9 bits). More tokens are merged, 8 sorted pieces at a time, each value
// finding its place by binary search (k_merge_lds, then k_merge). Other work-groups of these launches clear the table
// meanwhile, each launch a share of it. k_sums: a wavefront adds
// the rows of `len` places of the sorted list, 256 channels of them; a token whose
// rows lie within writes its sum to the table, the first and the last one's may go on
// beyond it, and are kept apart for k_join. Bound: HBM, the table's write.
#include <type_traits>

#include "ssd_common.h"
#include "ssd_internal.h"

namespace ssd {

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64, kSortKeys = 4, kBins = 512;
constexpr int kTileBits = 12;  // tokens of a sorted piece: 2^12 at most
static_assert(kSortThreads * kSortKeys == 1 << kTileBits, "a piece fits the registers");

// 4 consecutive values of a row at any alignment of their type; n of them where the row ends before that (zeros behind it).
constexpr int V = 4;
template <typename T>
__device__ __forceinline__ void load(float (&v)[V], const T *p, int n) {
    if (n >= V) {
        if constexpr (sizeof(T) == 2) {
            typedef uint32_t word __attribute__((ext_vector_type(2), aligned(2)));
            const word q = *reinterpret_cast<const word *>(p);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = __uint_as_float(e & 1 ? q[e >> 1] & 0xffff0000u : q[e >> 1] << 16);
        } else {
            typedef float word __attribute__((ext_vector_type(4), aligned(4)));
            const word q = *reinterpret_cast<const word *>(p);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = q[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = e < n ? (float)p[e] : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void store(T *p, const float (&v)[V], int n) {
    if (n >= V) {
        if constexpr (sizeof(T) == 2) {
            typedef uint32_t word __attribute__((ext_vector_type(2), aligned(2)));
            *reinterpret_cast<word *>(p) = __builtin_bit_cast(u32x2, bf16x4{(bf16)v[0], (bf16)v[1], (bf16)v[2], (bf16)v[3]});
        } else {
            typedef float word __attribute__((ext_vector_type(4), aligned(4)));
            *reinterpret_cast<word *>(p) = word{v[0], v[1], v[2], v[3]};
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < n) p[e] = (T)v[e];
    }
}

// 4 values a lane, 64 lanes to a slice of a row. Work-groups go over the rows' slices in turn.
template <typename TT, typename TY>
__global__ __launch_bounds__(256) void k_embed(const int *tokens, const TT *table, TY *y, float scale, int64_t rows, int vocab, int dim) {
    const int slices = (dim + 64 * V - 1) / (64 * V);
    const int64_t n = rows * slices, hop = (int64_t)gridDim.x * 4;
    const int lane = threadIdx.x & 63;
    for (int64_t k = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)); k < n; k += hop) {
        const int64_t r = k / slices;
        const int d = ((int)(k - r * slices) * 64 + lane) * V;
        if (d >= dim) continue;
        const int t = tokens[r];
        float v[V];
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = 0.f;
        if ((uint32_t)t < (uint32_t)vocab) {
            load(v, table + (int64_t)t * dim + d, dim - d);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] *= scale;
        }
        store(y + r * dim + d, v, dim - d);
    }
}

// A share of the table to clear: n16 pieces of 16 bytes, and `rest` of 2 behind them.
struct Share {
    u32x4 *p;
    int64_t n16;
    int rest;
};
template <int THREADS>
__device__ __forceinline__ void clear_share(const Share &c, int64_t block, int64_t blocks) {
    const int64_t i0 = block * THREADS + threadIdx.x;
    for (int64_t i = i0; i < c.n16; i += blocks * THREADS) __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, c.p + i);  // past the caches: nothing reads the table soon (71 -> 58 us)
    if (i0 < c.rest) reinterpret_cast<uint16_t *>(c.p + c.n16)[i0] = 0;
}

// Work-groups below `tiles` sort a piece of 2^bits tokens each: keys are
// token << bits | place in the piece, in order of their tokens; out: token << 32 | row.
// The others clear.
__global__ __launch_bounds__(kSortThreads) void k_sort(const int *tokens, uint64_t *out, int64_t rows, int vocab, int bits, int passes,
                                                       int digit, int tiles, Share clear) {
    if ((int)blockIdx.x >= tiles) {
        clear_share<kSortThreads>(clear, blockIdx.x - tiles, gridDim.x - tiles);
        return;
    }
    __shared__ uint32_t keys[kSortThreads * kSortKeys];
    __shared__ uint32_t count[kSortWaves][kBins];
    __shared__ uint32_t sums[kSortWaves];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t first = (int64_t)blockIdx.x << bits;
    const int n = (int)min((int64_t)1 << bits, rows - first);
    const int each = (n + kSortThreads - 1) / kSortThreads;  // keys of a lane, 64 places apart
    uint32_t key[kSortKeys];
#pragma unroll
    for (int e = 0; e < kSortKeys; ++e) {
        const int i = (w * each + e) * 64 + lane;
        key[e] = ~0u;  // behind every token
        if (e < each && i < n) {
            const uint32_t t = (uint32_t)tokens[first + i];
            key[e] = (t < (uint32_t)vocab ? t : (uint32_t)vocab) << bits | (uint32_t)i;
        }
    }
    const uint64_t below = ((uint64_t)1 << lane) - 1;
    const uint32_t bins = 1u << digit;
    for (int p = 0; p < passes; ++p) {
        const int shift = bits + p * digit;
        for (uint32_t i = threadIdx.x; i < kSortWaves * kBins; i += kSortThreads) (&count[0][0])[i] = 0;
        __syncthreads();
        // a key's place among its wavefront's keys of the same digit
        uint32_t place[kSortKeys];
#pragma unroll
        for (int e = 0; e < kSortKeys; ++e) {
            place[e] = 0;
            if (e < each) {
                const uint32_t d = (key[e] >> shift) & (bins - 1);
                uint64_t same = ~(uint64_t)0;
                for (int b = 0; b < digit; ++b) {
                    const int64_t one = -(int64_t)((d >> b) & 1);
                    same &= ~(__ballot(one != 0) ^ (uint64_t)one);
                }
                const uint32_t before = count[w][d];
                __builtin_amdgcn_wave_barrier();
                if ((same & below) == 0) count[w][d] = before + (uint32_t)__popcll(same);
                __builtin_amdgcn_wave_barrier();
                place[e] = before + (uint32_t)__popcll(same & below);
            }
        }
        __syncthreads();
        // the counts' exclusive sums, digit by digit and within it wavefront by wavefront: thread t takes
        // 8 wavefronts' counts of digit t / 2
        constexpr int kEach = kSortWaves * kBins / kSortThreads;
        const uint32_t dd = threadIdx.x / (kSortWaves / kEach), w0 = threadIdx.x % (kSortWaves / kEach) * kEach;
        uint32_t c[kEach], s = 0;
#pragma unroll
        for (int j = 0; j < kEach; ++j) c[j] = count[w0 + j][dd], s += c[j];
        uint32_t up = s;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t v = __shfl_up(up, o, 64);
            if (lane >= o) up += v;
        }
        if (lane == 63) sums[w] = up;
        __syncthreads();
        uint32_t base = up - s;
        for (int j = 0; j < w; ++j) base += sums[j];
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            count[w0 + j][dd] = base;
            base += c[j];
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kSortKeys; ++e)
            if (e < each) keys[count[w][(key[e] >> shift) & (bins - 1)] + place[e]] = key[e];
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kSortKeys; ++e)
            if (e < each) key[e] = keys[(w * each + e) * 64 + lane];
        __syncthreads();
    }
#pragma unroll
    for (int e = 0; e < kSortKeys; ++e) {
        const int i = (w * each + e) * 64 + lane;
        if (e < each && i < n) out[first + i] = (uint64_t)(key[e] >> bits) << 32 | (uint64_t)(first + (key[e] & ((1u << bits) - 1)));
    }
}

// The same for the first pieces' runs, where all 8 fit LDS as tokens (128 KB): a work-group takes 1024 places, and a step of its
// searches is one of LDS instead of the L2 (16384 tokens: 10 us with k_merge, 8 so). Between two runs the
// earlier one's rows go first where tokens are equal.
__global__ __launch_bounds__(1024) void k_merge_lds(const uint64_t *in, uint64_t *out, int64_t n, int run, int64_t blocks, Share clear) {
    if (blockIdx.x >= blocks) {
        clear_share<1024>(clear, blockIdx.x - blocks, gridDim.x - blocks);
        return;
    }
    __shared__ uint32_t tokens[8 << kTileBits];
    const int64_t first = (int64_t)blockIdx.x * 1024, group = first / (8 * run) * (8 * run);
    const int many = (int)min((int64_t)8 * run, n - group);
    for (int i0 = threadIdx.x; i0 < many; i0 += 8 * 1024) {  // 8 on their way
        uint64_t k[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) k[u] = i0 + u * 1024 < many ? in[group + i0 + u * 1024] : 0;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (i0 + u * 1024 < many) tokens[i0 + u * 1024] = (uint32_t)(k[u] >> 32);
    }
    __syncthreads();
    const int me = (int)(first - group) + (int)threadIdx.x;
    if (me >= many) return;
    const uint64_t v = in[group + me];
    const uint32_t t = (uint32_t)(v >> 32);
    const int mine = me / run;
    int at = me - mine * run;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (j == mine || j * run >= many) continue;
        int lo = 0, hi = min(run, many - j * run);
        while (lo < hi) {
            const int m = (lo + hi) >> 1;
            const uint32_t o = tokens[j * run + m];
            if (o < t || (o == t && j < mine)) lo = m + 1;
            else hi = m;
        }
        at += lo;
    }
    out[group + at] = v;
}

// Sorted runs of `run` values (the last one shorter) merged 8 at a time: a value's place is its own in its run
// and, of each other run, the number of values below it (no two are equal).
// Work-groups from `blocks` on clear.
__global__ __launch_bounds__(256) void k_merge(const uint64_t *in, uint64_t *out, int64_t n, int64_t run, int64_t blocks, Share clear) {
    if (blockIdx.x >= blocks) {
        clear_share<256>(clear, blockIdx.x - blocks, gridDim.x - blocks);
        return;
    }
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const uint64_t v = in[i];
    const int64_t mine = i / run * run, group = i / (8 * run) * (8 * run);
    int64_t at = group + (i - mine);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t b = group + j * run;
        if (b == mine || b >= n) continue;
        int64_t lo = 0, hi = min(run, n - b);
        while (lo < hi) {
            const int64_t m = (lo + hi) >> 1;
            if (in[b + m] < v) lo = m + 1;
            else hi = m;
        }
        at += lo;
    }
    out[at] = v;
}

// The row of the table that a token's sum goes to.
template <typename TG>
__device__ __forceinline__ void put(const EmbedBwdArgs &a, int64_t token, int d, float (&sum)[V]) {
    TG *p = reinterpret_cast<TG *>(a.dtable) + token * a.dim + d;
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] *= a.scale;
    if (a.accumulate) {
        float old[V];
        load(old, p, a.dim - d);
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] += old[e];
    }
    store(p, sum, a.dim - d);
}

template <typename TY, typename TG>
__global__ __launch_bounds__(64) void k_sums(EmbedBwdArgs a) {
    const int64_t piece = blockIdx.x;
    constexpr int U = 8;  // rows on their way (with 16, half the wavefronts: 1.5 us more of 54)
    const int d = ((int)blockIdx.y * 64 + (int)threadIdx.x) * V;
    const int64_t s = piece * a.len, end = min(s + a.len, a.rows);
    const bool live = d < a.dim;
    auto token = [&](int64_t i) { return (uint32_t)(a.sorted[i] >> 32); };
    uint32_t now = token(s);
    bool head = s > 0 && token(s - 1) == now;
    const uint32_t after = end < a.rows ? token(end) : ~0u;
    float sum[V];
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] = 0.f;
    auto flush = [&](bool tail) {
        if (!live || now >= (uint32_t)a.vocab) return;
        if (head || tail) store(a.part + (piece * 2 + (head ? 0 : 1)) * a.dim + d, sum, a.dim - d);
        else put<TG>(a, now, d, sum);
    };
    for (int64_t i = s; i < end; i += U) {
        float v[U][V];
        uint32_t t[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint64_t k = i + u < end ? a.sorted[i + u] : ~(uint64_t)0;
            t[u] = (uint32_t)(k >> 32);
#pragma unroll
            for (int e = 0; e < V; ++e) v[u][e] = 0.f;
            if (live && t[u] < (uint32_t)a.vocab) load(v[u], reinterpret_cast<const TY *>(a.dy) + (int64_t)(uint32_t)k * a.dim + d, a.dim - d);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i + u >= end) break;
            if (t[u] != now) {
                flush(false);
                now = t[u];
                head = false;
#pragma unroll
                for (int e = 0; e < V; ++e) sum[e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < V; ++e) sum[e] += v[u][e];
        }
    }
    flush(end < a.rows && after == now);
}

// The sums of a token whose rows begin in piece blockIdx.x and go on beyond it, in order.
// 4 wavefronts take a quarter of the pieces each.
template <typename TG>
__global__ __launch_bounds__(256, 8) void k_join(EmbedBwdArgs a) {
    __shared__ float share[4][64][V];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t p = blockIdx.x, s = p * a.len, end = s + a.len;  // never the last piece
    // all at once: one wait
    const int64_t after = (p + 1 + lane) * a.len;
    const uint64_t k0 = a.sorted[s > 0 ? s - 1 : 0], k1 = a.sorted[s], k2 = a.sorted[end - 1], k3 = a.sorted[end];
    uint64_t begins = a.sorted[after < a.rows ? after : 0];
    const uint64_t mine = k2 >> 32;
    if (mine >= (uint64_t)a.vocab || mine != k3 >> 32) return;
    if (mine == k1 >> 32 && s > 0 && mine == k0 >> 32) return;  // it began earlier
    // the pieces behind this one that begin with the token: it ends in the last of them
    int64_t pieces = 0;
    for (int64_t next = after;;) {
        const int n = __popcll(__ballot(next < a.rows && begins >> 32 == mine));
        pieces += n;
        if (n < 64) break;
        next += 64 * a.len;
        begins = a.sorted[next < a.rows ? next : 0];
    }
    const int64_t each = (pieces + 3) / 4;
    const int d = ((int)blockIdx.y * 64 + lane) * V;
    float sum[V];
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] = 0.f;
    if (d < a.dim) {
        if (w == 0) load(sum, a.part + (p * 2 + 1) * a.dim + d, a.dim - d);
        const int64_t to = min((w + 1) * each, pieces);
#pragma unroll 4
        for (int64_t q = w * each; q < to; ++q) {
            float v[V];
            load(v, a.part + (p + 1 + q) * 2 * a.dim + d, a.dim - d);
#pragma unroll
            for (int e = 0; e < V; ++e) sum[e] += v[e];
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) share[w][lane][e] = sum[e];
    __syncthreads();
    if (w == 0 && d < a.dim) {
#pragma unroll
        for (int k = 1; k < 4; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) sum[e] += share[k][lane][e];
        put<TG>(a, (int64_t)mine, d, sum);
    }
}

static ssd_status status_of(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_ERR_HIP; }
template <typename F>
static ssd_status pick_type(ssd_dtype t, F fn) {
    return t == SSD_BF16 ? fn(bf16{}) : fn(float{});
}

ssd_status launch_embed(const int *tokens, const void *table, void *y, float scale, int64_t rows, int64_t vocab, int64_t dim,
                        ssd_dtype dtype, ssd_dtype y_dtype, hipStream_t s) {
    return pick_type(dtype, [&](auto tt) {
        return pick_type(y_dtype, [&](auto ty) {
            using TT = decltype(tt);
            using TY = decltype(ty);
            const int64_t n = rows * ((dim + 64 * V - 1) / (64 * V)), blocks = (n + 3) / 4, most = 1 << 20;
            return status_of(launch(k_embed<TT, TY>, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), s, tokens, (const TT *)table,
                                    (TY *)y, scale, rows, (int)vocab, (int)dim));
        });
    });
}

EmbedPlan embed_plan(int64_t rows, int64_t vocab, int64_t dim) {
    EmbedPlan p = {};
    int bits = 0;
    while ((vocab >> bits) != 0) ++bits;  // of `vocab` itself, which stands for tokens outside the table
    p.passes = (bits + 8) / 9;
    p.digit = (bits + p.passes - 1) / p.passes;
    p.bits = 32 - bits < kTileBits ? 32 - bits : kTileBits;
    p.tiles = (rows + ((int64_t)1 << p.bits) - 1) >> p.bits;
    // pieces for 4 wavefronts a SIMD (38195 x 248 in fp32: 67 us with 1024 of them at most, 50 so), or 1024 where rows are long
    const int64_t slices = (dim + 64 * V - 1) / (64 * V), most = slices < 4 ? 4096 / slices : 1024;
    p.len = 16;
    while (p.len < 256 && rows / p.len > most) p.len *= 2;
    p.pieces = (rows + p.len - 1) / p.len;
    return p;
}

ssd_status launch_embed_bwd(EmbedBwdArgs a, const EmbedPlan &p, const int *tokens, uint64_t *one, uint64_t *two, ssd_dtype dy_dtype,
                            ssd_dtype dtype, hipStream_t s) {
    int merges = 0;
    for (int64_t run = (int64_t)1 << p.bits; run < a.rows; run *= 8) ++merges;
    // the table is cleared by shares of whole 16 bytes, one beside the sort and each merge
    const int64_t bytes = a.accumulate ? 0 : (int64_t)a.vocab * a.dim * (dtype == SSD_BF16 ? 2 : 4);
    const int64_t all = bytes / 16, each = (all + merges) / (merges + 1);
    auto share = [&](int k) {
        const int64_t from = k * each < all ? k * each : all, to = k < merges && from + each < all ? from + each : all;
        return Share{reinterpret_cast<u32x4 *>(a.dtable) + from, to - from, k == merges ? (int)(bytes % 16 / 2) : 0};
    };
    auto fill = [&](const Share &c, int64_t per) {  // work-groups, of `per` pieces of 16 bytes each, or up to 2048
        const int64_t n = (c.n16 + per - 1) / per;
        return n > 2048 ? 2048 : n > 0 ? n : c.rest ? 1 : 0;
    };
    Share c = share(0);
    const int64_t more = fill(c, 4 * kSortThreads);
    if (p.tiles + more == 0) return SSD_OK;
    ssd_status st = status_of(launch(k_sort, dim3((unsigned)(p.tiles + more)), dim3(kSortThreads), s, tokens, one, a.rows, a.vocab, p.bits,
                                     p.passes, p.digit, (int)p.tiles, c));
    if (st != SSD_OK || a.rows == 0) return st;
    for (int k = 1; k <= merges; ++k) {
        c = share(k);
        const int64_t run = ((int64_t)1 << p.bits) << (3 * (k - 1));
        if (k == 1) {
            const int64_t blocks = (a.rows + 1023) / 1024;
            st = status_of(launch(k_merge_lds, dim3((unsigned)(blocks + fill(c, 4 * 1024))), dim3(1024), s, one, two, a.rows, (int)run, blocks, c));
        } else {
            const int64_t blocks = (a.rows + 255) / 256;
            st = status_of(launch(k_merge, dim3((unsigned)(blocks + fill(c, 4 * 256))), dim3(256), s, one, two, a.rows, run, blocks, c));
        }
        if (st != SSD_OK) return st;
        uint64_t *t = one;
        one = two;
        two = t;
    }
    a.sorted = one;
    a.len = p.len;
    const unsigned slices = (unsigned)((a.dim + 64 * V - 1) / (64 * V));
    return pick_type(dy_dtype, [&](auto ty) {
        return pick_type(dtype, [&](auto tg) {
            using TY = decltype(ty);
            using TG = decltype(tg);
            const ssd_status e = status_of(launch(k_sums<TY, TG>, dim3((unsigned)p.pieces, slices), dim3(64), s, a));
            if (e != SSD_OK || p.pieces < 2) return e;
            return status_of(launch(k_join<TG>, dim3((unsigned)(p.pieces - 1), slices), dim3(256), s, a));
        });
    });
}

}  // namespace ssd
