// Internal interfaces between the C ABI host code and the kernel files.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssd.h"

namespace ssd {

// Everything the forward launch sequence needs, validated by the caller.
struct FwdArgs {
    const void *X, *dt, *B, *C;
    const float *A, *D;
    void *Y;
    float *final_state;        // may be null
    const float *init;         // (batch, H, P, N) initial state, or null for zero
    int64_t batch, T, H, P, N, G, Q, nC, Tpad;
    const int *cu;             // packed variable-length batch: (batch + 1) cumulative lengths, or null
    int64_t total;             // tokens in the packed batch (cu != null)
    const float *dt_bias;      // fused prologue: dt = [softplus](dt + dt_bias[h]); null = no bias
    int softplus;
    const void *z;             // fused epilogue: Y *= silu(z), z shaped like X; null = no gate
    const float *conv_w;       // fused input activation: X <- silu(causal conv of X), taps (H P, 4); null = none
    const float *conv_b;       // its bias (H P), or null (zero)
    ssd_dtype dtype;
    float *cs2, *dtf;          // workspace: (batch, H, Tpad) each
    void *Gbuf;                // workspace: (batch, G, Tpad / tt, tt, tt) in the storage type
    int64_t g_bytes;
    int ns, tt;                // walk plan: work-groups per head, tile tokens
    int S, cps;                // walk plan: sequence segments, chunks per segment
    int segk;                  // walk plan: pre-pass sub-segments per segment (1 or 2)
    float *seg;                // workspace: (batch, H, (S - 1) segk, P, N) fp32 (sub-)segment states
    bool no_g;                 // the caller reads no C B^T tiles (the backward): prepare skips them
};

// How the walk covers a shape: ns work-groups per head (P / ns columns each)
// and tiles of tt tokens.
struct WalkPlan {
    int ns, tt;   // work-groups per head (P / ns columns each), tile tokens
    int S, cps;   // sequence segments walked in parallel, chunks per segment
    int segk;     // sub-segments per segment in the end-state pre-pass (1 or 2)
};
// Fills the plan; -1 if no kernel covers the shape.
// segments: whether the sequence may be split (not for packed batches).
int fwd_plan(ssd_dtype dt, int64_t batch, int64_t H, int64_t P, int64_t N, int64_t Q, int64_t nC,
             bool segments, WalkPlan *plan);

// Kernel arguments of the chunk walk (passed by value).
struct PrepArgs {
    const void *dt, *B, *C;
    const float *A;
    void *Gbuf;
    float *cs2, *dtf;
    int T, H, G, nC, Tpad, ntiles, cb_blocks;
    const int *cu;             // see FwdArgs
    int total;
    const float *dt_bias;      // see FwdArgs
    int softplus;
    uint32_t g_bytes;
};

struct WalkArgs {
    const void *X, *B, *C;
    void *Y;
    const void *Gbuf;
    const float *cs2, *dtf, *D;
    const float *init;         // (batch, H, P, N) or null for a zero state
    float *final_state;        // may be null
    int batch, T, H, G, nC, Tpad;
    int P, NS;                 // head dimension, and the work-groups sharing each head's P columns
    int S, SL, cps;            // sequence segments, segments in this launch, chunks per segment
    int segk;                  // seg holds (S - 1) segk sub-segment states per (batch, head); segment
                               // s > 0 enters with the one in slot s segk - 1
    float *seg;                // (batch, H, (S - 1) segk, P, N) segment states (S > 1)
    const int *cu;             // see FwdArgs
    int total;
    const void *z;             // see FwdArgs
    const float *conv_w, *conv_b;  // see FwdArgs
    uint32_t g_bytes;
};

struct StepArgs {
    float *state;
    const void *x, *dt, *B, *C;
    const float *A, *D;
    void *y;
    const float *dt_bias;      // see FwdArgs
    int softplus;
    const void *z;             // (batch, H, P) like x, or null
    void *conv_state;          // input convolution: (batch, H P, 3) raw inputs, oldest first, storage type
    const float *conv_w;       // its taps (H P, 4), or null for no convolution
    const float *conv_b;       // its bias (H P), or null (zero)
    int64_t batch, H, P, N, G;
    ssd_dtype dtype;
    // beam search: row b's state (and conv state) comes from row parent[b] of
    // state_in (conv_in), of which there are src_rows; null for a step in place
    const int *parent;
    const float *state_in;
    const void *conv_in;
    int64_t src_rows;
};

// Backward pass (ssd_bwd.hip).
struct StatePassArgs {          // k_state_pass
    const void *U, *V;          // X / dY (batch, T, H, P) and B / C (batch, T, G, N)
    const float *cs2, *dtf;     // log-decay workspace (batch, H, Tpad)
    const float *init;          // state before the first tile walked (fp32), or null
    void *Sst;                  // (batch, H, ntiles, P, N) storage type: the state entering each tile
    float *out;                 // state after the last tile walked (fp32), or null
    int H, G, T, Tpad, ntiles, tpc;  // tpc: 64-token tiles per chunk
};

struct BwdTileArgs {            // k_bwd_tile
    const void *X, *dY, *B, *C, *dt;
    const float *D;
    const void *Hst, *Est;      // entering states / arriving adjoints per tile
    const float *cs2, *dtf;
    void *dX;
    float *rbuf, *qbuf, *xybuf; // per (batch, head, token): x.v, dy.y' - dt x.v, dy.x
    float *dBp, *dCp;           // (batch, Tpad, nblk, G, N) partial sums over head blocks
    void *dB, *dC;              // one head block per group: dB, dC (storage type) written directly
    float *lamb;                // (batch, H, ntiles, NS, 8) per-wavefront shares of
                                // <E_tile, state after the tile>
    float *dXp;                 // NS > 1: (NS, batch, T, H, P) fp32 parts of dX
    size_t tok_stride;          // elements between the n slices' rbuf / qbuf parts
    size_t dx_stride;           // elements between the n slices' dXp parts
    int H, G, T, Tpad, ntiles, tpc, nblk;
};

struct BwdFinArgs {             // k_bwd_fin
    const float *qbuf, *rbuf, *xybuf, *lamb;
    size_t tok_stride;          // elements between the n slices' rbuf / qbuf parts
    int ns;                     // n slices of k_bwd_tile
    const void *dt;
    const float *A;
    void *ddt;
    float *dApart, *dDpart;     // (batch, H, ntiles) shares of dA, dD
    int batch, T, Tpad, H, ntiles;
};

struct BwdArgs {
    FwdArgs f;                  // forward inputs and the prepared log-decays
    const void *dY;
    const float *dF;            // gradient of the final state, or null
    void *dX, *ddt, *dB, *dC;
    float *dA, *dD, *dinit;     // dinit may be null
    void *Hst, *Est;            // workspace, storage type
    float *lamb, *dApart, *dDpart;                  // workspace, fp32, (batch, H, ntiles) each
    float *rbuf, *qbuf, *xybuf, *dBp, *dCp;          // workspace, fp32 (rbuf, qbuf: one part per n slice)
    float *dXp;                 // workspace, fp32, n slices > 1 only
    int nblk;                   // head blocks per group
};

// Whether a backward kernel covers (dtype, P, N).
bool bwd_supported(ssd_dtype dt, int64_t P, int64_t N);
// Work-groups k_bwd_tile splits the n axis over (1 where it fits one CU's LDS).
int bwd_nslices(ssd_dtype dt, int64_t P, int64_t N);
// The backward launches (after launch_prepare on the same FwdArgs).
ssd_status launch_bwd(const BwdArgs &w, hipStream_t s);

// Phase 1: chunk-local log-decay prefix sums and (unless f.no_g) C B^T tiles
// into the workspace.
ssd_status launch_prepare(const FwdArgs &f, hipStream_t s);
// Whether the walk with the fused input convolution fits LDS for a column slice.
bool walk_conv_fits(ssd_dtype dt, int64_t Q, int64_t PW, int64_t N);
// Phase 2: the chunk walk (reads the prepared workspace).
ssd_status launch_walk(const FwdArgs &f, hipStream_t s);
// The walk with the fused input convolution (f.conv_w set; ssd_walk_conv.hip).
ssd_status launch_walk_conv(const FwdArgs &f, hipStream_t s);
// The walk with the state kept in the wavefronts that update it
// (ssd_walk_rs.hip): bf16 storage, 64-token tiles, column slices of 32 or 64
// and N of 64 or 128, with or without the gate and the input convolution.
bool walk_rs_supported(const FwdArgs &f);
ssd_status launch_walk_rs(const FwdArgs &f, hipStream_t s);
// The end states of a split sequence's segments 0 .. S - 2 (each entered with
// zero, the first with f.init) into f.seg (ssd_seg_states.hip).
ssd_status launch_seg_states(const FwdArgs &f, hipStream_t s);
// RMS norm (ssd_norm.hip). rows counts (row, group) pairs of Dg values each.
struct NormArgs {
    const void *x, *res;        // res may be null: no residual
    const float *w;             // (groups, Dg)
    void *res_out, *y;          // y null where q is given
    uint8_t *q, *scale;         // 8-bit output, or null
    float *rstd;                // (rows) or null
    int64_t rows, groups;
    int Dg;
    float eps;
    ssd_dtype dtype, res_dtype;
};
ssd_status launch_rms_norm(const NormArgs &a, hipStream_t s);
ssd_status launch_mx_quantize(const void *x, uint8_t *q, uint8_t *scale, int64_t n, ssd_dtype dtype, hipStream_t s);

struct NormBwdArgs {
    const void *dy, *h, *dres;  // dres may be null
    const float *w, *rstd;      // rstd (rows, groups)
    void *dx, *dh;              // dh may be null; written where h's type is not dy's
    float *dw;
    float *part;                // workspace: (nb, groups, Dg)
    int64_t rows, groups;
    int Dg, nb;
    ssd_dtype dtype, res_dtype;
};
int norm_bwd_blocks(int64_t rows, int64_t groups, int64_t n);
ssd_status launch_rms_norm_bwd(const NormBwdArgs &a, hipStream_t s);

// out[d] = sum over b < nb of part[b][d], in a fixed order (fp32).
ssd_status launch_column_sums(const float *part, float *out, int nb, int64_t D, hipStream_t s);

// Matrix products (ssd_linear.hip): y (M x N) = act(x w^T + bias) + res.
struct LinearArgs {
    const void *x, *w;          // rows of ldx / ldw bytes (multiples of 4; few rows: of the type), kbytes of them along k
    const uint8_t *xscale, *wscale;  // 8-bit operands: a scale for each 32 along k, rows of lds bytes
    const float *xs, *ws;       // 8-bit integers: a scale for each row of x and of w
    int64_t ldx, ldw, lds;
    const float *bias;          // (N) or null
    const void *res;            // (M x N) or null
    void *y, *pre;              // pre: z before the activation, or null
    float *part;                // workspace: (splits, part_stride) where the sum over k is split
    int M, N, act;
    uint32_t kbytes;
    bool xt, wt;                // bf16: x (w) is given as (krows x M) ((krows x N)), rows along k
    int krows;
    int nm, nn, steps, splits, steps_per_split;
    int64_t ldy;                // values from one row of y, res and pre to the next (0: N)
    bool whole;                 // set at launch: groups of 4 columns are whole and aligned
};
// Floats from one part of a split sum to the next.
__host__ __device__ inline int64_t part_stride(int64_t M, int64_t N) { return (M * N + 3) & ~(int64_t)3; }
struct LinearPlan {
    int bm, bn;                 // a work-group's tile of y; 0: the few-rows kernel
    int nm, nn;                 // tiles
    int steps, splits, steps_per_split;
    int n_main;                 // > 0: this plan is for the first n_main columns, the next for the rest
    int rest_bm, rest_bn, rest_nm, rest_nn;
};
// along_k: an operand has its rows along k (the few-rows kernel takes none of these).
LinearPlan linear_plan(int64_t M, int64_t N, int64_t kbytes, bool f32, bool along_k);
ssd_status launch_linear(LinearArgs a, const LinearPlan &p, bool mx, ssd_dtype dtype, hipStream_t s);
// Two operands' rows (R2 may be 0) of n values of es bytes to rows of ldo values.
ssd_status launch_pad(const void *in1, void *out1, int64_t R1, const void *in2, void *out2, int64_t R2, int64_t n,
                      int64_t ldo, int es, hipStream_t s);
// fp32 only.
ssd_status launch_transpose(const void *in, void *out, int64_t R, int64_t C, int64_t ldo, hipStream_t s);
// dz (null: not wanted) and the shares of db, of dz_rows rows each (null: not wanted).
int dz_rows(int64_t M, int64_t ldz);
ssd_status launch_dz(const void *dy, const void *pre, int act, void *dz, float *part, int64_t M, int64_t N, int64_t ldz,
                     ssd_dtype dtype, hipStream_t s);

// Beam search's selection (ssd_beam.hip).
struct BeamArgs {
    const void *logits;         // (rows, V), rows = batch x beams
    const float *scores;        // (rows)
    const uint8_t *finished;    // (rows) or null
    float *out_scores;
    int *parent, *token;
    uint8_t *out_finished;      // or null
    uint64_t *keys;             // workspace: (rows, lists, beams)
    double *sums;               // workspace: (rows, lists) sums of exponentials, relative to the first key's logit
    int64_t rows;
    int beams, V, eos, lists, tiles;
};
void beam_plan(int64_t V, int *lists, int *tiles);
ssd_status launch_beam_select(const BeamArgs &a, int64_t batch, ssd_dtype dtype, hipStream_t s);

// Gated linear recurrence (ssd_gated.hip).
struct GatedArgs {
    const void *x, *f, *i, *dy;  // i: null where the input is not gated; dy: the backward's
    int64_t ldx, ldf, ldi;       // values from one token to the next
    const uint8_t *reset;        // (batch, T) or null
    const float *rate;           // (D), decay "rate" only
    const float *init, *dfinal;  // (batch, D) or null
    float *states;               // (batch, nchunks, D): written by the forward (or null), read by the backward
    void *y, *dx, *df, *di;
    float *final, *dinit, *drate;
    float *part;                 // backward: shares of drate, (batch, nchunks, D)
    int64_t batch, T, D, nchunks;
    int cols;                    // pieces of 64 channels
    uint32_t wide, share, tickets;  // a chunk's tiles of all columns and sequences, how many a ticket is for, tickets a chunk
    uint32_t *ticket;            // workspace, cleared before: the next chunk to take; per (batch, chunk, column) ...
    uint64_t *pieces;            // ... its decay and its own state's end,
    uint32_t *ends;              // ... and the state behind it
};
struct GatedPlan {
    bool fits;
    int64_t cols, nchunks, tiles;  // pieces of 64 channels, chunks, and chunks of all sequences and columns
    int64_t share, groups;         // a chunk's tiles of a ticket, and work-groups
    int64_t word_bytes;            // workspace of either pass
    int64_t rate_bytes;            // the backward's, behind that, for the rates' gradient
};
GatedPlan gated_plan(int64_t batch, int64_t T, int64_t D, ssd_dtype dtype, bool backward);
ssd_status launch_gated_fwd(GatedArgs a, const GatedPlan &p, ssd_dtype dtype, int decay, void *workspace, hipStream_t s);
ssd_status launch_gated_bwd(GatedArgs a, const GatedPlan &p, ssd_dtype dtype, int decay, void *workspace, hipStream_t s);
struct GatedStepArgs {
    const float *state_in;
    float *state_out;
    const int *parent;           // (rows), or null: each row's own
    int64_t src;
    const void *x, *f, *i;
    int64_t ldx, ldf, ldi;
    const float *rate;
    void *y;
    int64_t rows, D;
};
ssd_status launch_gated_step(const GatedStepArgs &a, ssd_dtype dtype, int decay, hipStream_t s);

// Embedding (ssd_embed.hip).
ssd_status launch_embed(const int *tokens, const void *table, void *y, float scale, int64_t rows, int64_t vocab, int64_t dim,
                        ssd_dtype dtype, ssd_dtype y_dtype, hipStream_t s);
struct EmbedPlan {
    int bits, passes, digit;     // tokens of a sorted piece (2^bits), and the sort's digits
    int64_t tiles;               // sorted pieces
    int len;                     // rows of a piece of sums
    int64_t pieces;
};
EmbedPlan embed_plan(int64_t rows, int64_t vocab, int64_t dim);
struct EmbedBwdArgs {
    const void *dy;              // (rows, dim)
    void *dtable;                // (vocab, dim)
    const uint64_t *sorted;      // token << 32 | row
    float *part;                 // workspace: (pieces, 2, dim): a piece's first sum where it began earlier, its last where it goes on
    int64_t rows;
    int vocab, dim, len, accumulate;
    float scale;
};
// one, two: workspace of rows each (two: only where there are several sorted pieces)
ssd_status launch_embed_bwd(EmbedBwdArgs a, const EmbedPlan &p, const int *tokens, uint64_t *one, uint64_t *two, ssd_dtype dy_dtype,
                            ssd_dtype dtype, hipStream_t s);

// Logits before the choice (ssd_logits.hip).
struct LogitsArgs {
    const void *logits;
    void *out;
    const int *tokens, *lengths, *prompt;                 // tokens (rows, capacity); null where not given
    const float *repetition, *presence, *frequency;       // (rows) or null
    const float *bias;                                    // (bias_rows, vocab) or null
    const uint32_t *mask;                                 // (mask_rows, words) or null
    int64_t rows, vocab, capacity, words, bias_rows, mask_rows;
    int slices;
};
int64_t logits_slices(int64_t vocab);
ssd_status launch_logits(LogitsArgs a, ssd_dtype dtype, hipStream_t s);

// 8-bit integers (ssd_int.hip; the products: ssd_linear_int.hip).
ssd_status launch_int_quantize(const void *x, int8_t *q, float *scale, int64_t rows, int64_t dim, ssd_dtype dtype, hipStream_t s);
ssd_status launch_linear_int(const LinearArgs &a, const LinearPlan &p, ssd_dtype dtype, hipStream_t s);

// One recurrent decode step.
ssd_status launch_step(const StepArgs &a, hipStream_t s);

// Whether [a, a + na) and [b, b + nb) share a byte (a NULL one does not).
inline bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
    const uintptr_t pa = (uintptr_t)a, pb = (uintptr_t)b;
    return a && b && na > 0 && nb > 0 && pa < pb + (uintptr_t)nb && pb < pa + (uintptr_t)na;
}

// Launches a kernel and returns the status of that launch itself (not an
// error some earlier, unrelated runtime call may have left pending).
// A launch has fewer than 2^32 threads along a dimension. HIP refuses some of those beyond and
// cuts others down without a word, so callers with more rows than that launch them in slices,
// and a larger grid is refused here.
constexpr int64_t kMostThreads = UINT32_MAX;
template <typename T> struct ident { using type = T; };
template <typename... Args>
inline hipError_t launch(void (*kernel)(Args...), dim3 grid, dim3 block, hipStream_t s,
                         typename ident<Args>::type... args) {
    if ((int64_t)grid.x * block.x > kMostThreads || (int64_t)grid.y * block.y > kMostThreads) return hipErrorInvalidConfiguration;
    void *argv[] = {(void *)&args..., nullptr};
    return hipLaunchKernel((const void *)kernel, grid, block, argv, 0, s);
}

}  // namespace ssd
