// C ABI of libssd, continued: the gated linear recurrence, and a decoder's ends
// (embedding, logits) and projections from 8-bit integers. Every check runs on the host before
// anything is enqueued.
#include <stddef.h>
#include <stdint.h>

#include "ssd_common.h"
#include "ssd_internal.h"

namespace {

template <typename... P>
bool misaligned(const P *...p) {
    return (... || (((uintptr_t)p & 15u) != 0));
}

bool valid_dtype(int d) { return d == SSD_F32 || d == SSD_BF16; }

int64_t align256(int64_t v) { return (v + 255) & ~(int64_t)255; }

int64_t esize(ssd_dtype d) { return d == SSD_BF16 ? 2 : 4; }

ssd_status check_workspace(int64_t need, const void *workspace, size_t workspace_bytes) {
    if (need == 0) return SSD_OK;
    if (!workspace || workspace_bytes < (size_t)need) return SSD_ERR_WORKSPACE;
    return ((uintptr_t)workspace & 255u) ? SSD_ERR_ALIGN : SSD_OK;
}

// Whether an output lies on an input, or on another output. Bytes of each behind its address.
struct Span {
    const void *p;
    int64_t bytes;
};
template <size_t O, size_t I>
bool any_overlap(const Span (&out)[O], const Span (&in)[I]) {
    for (size_t k = 0; k < O; ++k) {
        for (const Span &i : in)
            if (ssd::overlap(out[k].p, out[k].bytes, i.p, i.bytes)) return true;
        for (size_t j = 0; j < k; ++j)
            if (ssd::overlap(out[k].p, out[k].bytes, out[j].p, out[j].bytes)) return true;
    }
    return false;
}

__global__ void k_copy_or_clear(const float *from, float *to, int64_t n) {
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) to[i] = from ? from[i] : 0.f;
}
ssd_status copy_or_clear(const float *from, float *to, int64_t n, hipStream_t s) {
    if (!to || n == 0 || from == to) return SSD_OK;
    const int64_t blocks = (n + 255) / 256, most = 1 << 16;
    return ssd::launch(k_copy_or_clear, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), s, from, to, n) == hipSuccess
               ? SSD_OK
               : SSD_ERR_HIP;
}

constexpr int64_t kMostDim = (int64_t)1 << 20;

ssd_status check_gated(int64_t batch, int64_t seqlen, int64_t dim, int decay, int dtype) {
    if (!valid_dtype(dtype) || decay < SSD_DECAY_LOG || decay > SSD_DECAY_RATE) return SSD_ERR_UNSUPPORTED;
    if (batch < 0 || seqlen < 0 || dim <= 0) return SSD_ERR_SHAPE;
    if (dim > kMostDim || seqlen > INT32_MAX || batch > INT32_MAX / dim) return SSD_ERR_UNSUPPORTED;
    return ssd::gated_plan(batch, seqlen, dim, (ssd_dtype)dtype, false).fits ? SSD_OK : SSD_ERR_UNSUPPORTED;
}

// The inputs of a recurrence, `rows` tokens of them: present, far enough apart, aligned to their type.
ssd_status check_tokens(const void *x, int64_t ldx, const void *f, int64_t ldf, const void *in_gate, int64_t ldi, int64_t dim,
                        int64_t es) {
    if (ldx < dim || ldf < dim || (in_gate && ldi < dim)) return SSD_ERR_SHAPE;
    constexpr int64_t most = (int64_t)1 << 22;  // a chunk's 128 tokens within 2^31 bytes
    if (ldx > most || ldf > most || (in_gate && ldi > most)) return SSD_ERR_UNSUPPORTED;
    if (((uintptr_t)x | (uintptr_t)f | (uintptr_t)in_gate) & (uintptr_t)(es - 1)) return SSD_ERR_ALIGN;
    return SSD_OK;
}
int64_t span(int64_t rows, int64_t ld, int64_t dim, int64_t es) { return rows > 0 ? ((rows - 1) * ld + dim) * es : 0; }

int64_t chunks(int64_t seqlen) { return (seqlen + SSD_GATED_CHUNK - 1) / SSD_GATED_CHUNK; }

}  // namespace

extern "C" {

size_t ssd_gated_scan_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, ssd_dtype dtype) {
    if (check_gated(batch, seqlen, dim, SSD_DECAY_LOG, (int)dtype) != SSD_OK) return (size_t)-1;
    return (size_t)ssd::gated_plan(batch, seqlen, dim, dtype, false).word_bytes;
}

ssd_status ssd_gated_scan_fwd(const void *x, int64_t ldx, const void *f, int64_t ldf, const void *in_gate, int64_t ldi,
                              int decay, const float *rate, const uint8_t *reset, const float *initial_state, void *y,
                              float *final_state, float *states, int64_t batch, int64_t seqlen, int64_t dim,
                              ssd_dtype dtype, void *workspace, size_t workspace_bytes, void *stream) {
    const bool empty = batch == 0 || seqlen == 0;
    if (!empty && (!x || !f || !y || (decay == SSD_DECAY_RATE && !rate))) return SSD_ERR_NULL;
    ssd_status st = check_gated(batch, seqlen, dim, decay, (int)dtype);
    if (st != SSD_OK) return st;
    if (decay != SSD_DECAY_RATE && rate) return SSD_ERR_UNSUPPORTED;
    const int64_t rows = batch * seqlen, es = esize(dtype);
    if ((st = check_tokens(x, ldx, f, ldf, in_gate, ldi, dim, es)) != SSD_OK) return st;
    if (misaligned((const char *)y, (const char *)rate, (const char *)reset, (const char *)initial_state,
                   (const char *)final_state, (const char *)states))
        return SSD_ERR_ALIGN;
    const ssd::GatedPlan plan = ssd::gated_plan(batch, seqlen, dim, dtype, false);
    if ((st = check_workspace(plan.word_bytes, workspace, workspace_bytes)) != SSD_OK) return st;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const int64_t nb = batch * dim * 4;
    if (any_overlap({{y, rows * dim * es}, {final_state, nb}, {states, nb * chunks(seqlen)}},
                    {{x, span(rows, ldx, dim, es)}, {f, span(rows, ldf, dim, es)}, {in_gate, span(rows, ldi, dim, es)},
                     {rate, dim * 4}, {reset, rows}, {initial_state, nb}}))
        return SSD_ERR_UNSUPPORTED;
    if (empty) return copy_or_clear(initial_state, final_state, batch * dim, s);
    ssd::GatedArgs a = {};
    a.x = x; a.f = f; a.i = in_gate; a.ldx = ldx; a.ldf = ldf; a.ldi = ldi; a.reset = reset; a.rate = rate;
    a.init = initial_state; a.states = states; a.y = y; a.final = final_state; a.batch = batch; a.T = seqlen; a.D = dim;
    a.nchunks = chunks(seqlen);
    return ssd::launch_gated_fwd(a, plan, dtype, decay, workspace, s);
}

size_t ssd_gated_scan_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int decay, ssd_dtype dtype) {
    if (check_gated(batch, seqlen, dim, decay, (int)dtype) != SSD_OK) return (size_t)-1;
    const ssd::GatedPlan p = ssd::gated_plan(batch, seqlen, dim, dtype, true);
    return (size_t)(p.word_bytes + (decay == SSD_DECAY_RATE ? p.rate_bytes : 0));
}

ssd_status ssd_gated_scan_bwd(const void *dy, const void *x, int64_t ldx, const void *f, int64_t ldf, const void *in_gate,
                              int64_t ldi, int decay, const float *rate, const uint8_t *reset, const float *states,
                              const float *d_final_state, void *dx, void *df, void *d_in_gate, float *drate,
                              float *d_initial_state, int64_t batch, int64_t seqlen, int64_t dim, ssd_dtype dtype,
                              void *workspace, size_t workspace_bytes, void *stream) {
    const bool empty = batch == 0 || seqlen == 0, has_rate = decay == SSD_DECAY_RATE;
    if (!empty && (!dy || !x || !f || !states || !dx || !df || (!in_gate != !d_in_gate) || (has_rate && !rate))) return SSD_ERR_NULL;
    if (has_rate && !drate) return SSD_ERR_NULL;
    ssd_status st = check_gated(batch, seqlen, dim, decay, (int)dtype);
    if (st != SSD_OK) return st;
    if (!has_rate && (rate || drate)) return SSD_ERR_UNSUPPORTED;
    const int64_t rows = batch * seqlen, es = esize(dtype);
    if ((st = check_tokens(x, ldx, f, ldf, in_gate, ldi, dim, es)) != SSD_OK) return st;
    if (misaligned((const char *)dy, (const char *)rate, (const char *)reset, (const char *)states, (const char *)d_final_state,
                   (const char *)dx, (const char *)df, (const char *)d_in_gate, (const char *)drate, (const char *)d_initial_state))
        return SSD_ERR_ALIGN;
    const ssd::GatedPlan plan = ssd::gated_plan(batch, seqlen, dim, dtype, true);
    const int64_t need = plan.word_bytes + (has_rate ? plan.rate_bytes : 0);
    if ((st = check_workspace(need, workspace, workspace_bytes)) != SSD_OK) return st;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const int64_t nb = batch * dim * 4, n = rows * dim * es;
    if (any_overlap({{dx, n}, {df, n}, {d_in_gate, n}, {drate, dim * 4}, {d_initial_state, nb}},
                    {{dy, n}, {x, span(rows, ldx, dim, es)}, {f, span(rows, ldf, dim, es)}, {in_gate, span(rows, ldi, dim, es)},
                     {rate, dim * 4}, {reset, rows}, {states, nb * chunks(seqlen)}, {d_final_state, nb}}))
        return SSD_ERR_UNSUPPORTED;
    if (empty) {
        if ((st = copy_or_clear(nullptr, drate, dim, s)) != SSD_OK) return st;
        return copy_or_clear(d_final_state, d_initial_state, batch * dim, s);
    }
    ssd::GatedArgs a = {};
    a.x = x; a.f = f; a.i = in_gate; a.dy = dy; a.ldx = ldx; a.ldf = ldf; a.ldi = ldi; a.reset = reset; a.rate = rate;
    a.dfinal = d_final_state; a.states = const_cast<float *>(states); a.dx = dx; a.df = df; a.di = d_in_gate;
    a.dinit = d_initial_state; a.drate = drate; a.batch = batch; a.T = seqlen; a.D = dim; a.nchunks = chunks(seqlen);
    return ssd::launch_gated_bwd(a, plan, dtype, decay, workspace, s);
}

ssd_status ssd_gated_step(const float *state_in, float *state_out, const int32_t *parent, int64_t src_rows, const void *x,
                          int64_t ldx, const void *f, int64_t ldf, const void *in_gate, int64_t ldi, int decay,
                          const float *rate, void *y, int64_t rows, int64_t dim, ssd_dtype dtype, void *stream) {
    if (rows != 0 && (!state_out || !x || !f || !y || (src_rows != 0 && !state_in) || (decay == SSD_DECAY_RATE && !rate)))
        return SSD_ERR_NULL;
    if (!valid_dtype((int)dtype) || decay < SSD_DECAY_LOG || decay > SSD_DECAY_RATE) return SSD_ERR_UNSUPPORTED;
    if (decay != SSD_DECAY_RATE && rate) return SSD_ERR_UNSUPPORTED;
    if (rows < 0 || dim <= 0 || src_rows < 0 || (!parent && src_rows < rows)) return SSD_ERR_SHAPE;
    if (dim > kMostDim || rows > INT32_MAX / dim || src_rows > INT32_MAX) return SSD_ERR_UNSUPPORTED;
    const int64_t es = esize(dtype);
    ssd_status st = check_tokens(x, ldx, f, ldf, in_gate, ldi, dim, es);
    if (st != SSD_OK) return st;
    if (misaligned((const char *)state_in, (const char *)state_out, (const char *)parent, (const char *)rate, (const char *)y))
        return SSD_ERR_ALIGN;
    if (rows == 0) return SSD_OK;
    const bool in_place = !parent && state_in == state_out;
    if (any_overlap({{state_out, rows * dim * 4}, {y, rows * dim * es}},
                    {{in_place ? nullptr : state_in, src_rows * dim * 4}, {parent, rows * 4}, {x, span(rows, ldx, dim, es)},
                     {f, span(rows, ldf, dim, es)}, {in_gate, span(rows, ldi, dim, es)}, {rate, dim * 4}}) ||
        ssd::overlap(y, rows * dim * es, state_in, src_rows * dim * 4))
        return SSD_ERR_UNSUPPORTED;
    ssd::GatedStepArgs a = {};
    a.state_in = state_in; a.state_out = state_out; a.parent = parent; a.src = src_rows; a.x = x; a.f = f; a.i = in_gate;
    a.ldx = ldx; a.ldf = ldf; a.ldi = ldi; a.rate = rate; a.y = y; a.rows = rows; a.D = dim;
    return ssd::launch_gated_step(a, dtype, decay, reinterpret_cast<hipStream_t>(stream));
}

static ssd_status check_embed(int64_t rows, int64_t vocab, int64_t dim) {
    if (rows < 0 || vocab <= 0 || dim <= 0) return SSD_ERR_SHAPE;
    return rows > INT32_MAX || vocab > kMostDim || dim > kMostDim ? SSD_ERR_UNSUPPORTED : SSD_OK;
}

ssd_status ssd_embedding(const int32_t *tokens, const void *table, float scale, void *y, int64_t rows, int64_t vocab,
                         int64_t dim, ssd_dtype dtype, ssd_dtype y_dtype, void *stream) {
    if (rows != 0 && (!tokens || !table || !y)) return SSD_ERR_NULL;
    if (!valid_dtype((int)dtype) || !valid_dtype((int)y_dtype)) return SSD_ERR_UNSUPPORTED;
    const ssd_status st = check_embed(rows, vocab, dim);
    if (st != SSD_OK) return st;
    if (misaligned((const char *)tokens, (const char *)table, (const char *)y)) return SSD_ERR_ALIGN;
    if (rows == 0) return SSD_OK;
    if (any_overlap({{y, rows * dim * esize(y_dtype)}}, {{tokens, rows * 4}, {table, vocab * dim * esize(dtype)}})) return SSD_ERR_UNSUPPORTED;
    return ssd::launch_embed(tokens, table, y, scale, rows, vocab, dim, dtype, y_dtype, reinterpret_cast<hipStream_t>(stream));
}

// Workspace of the gradient: the sorted tokens (twice where they are merged), then the pieces' open sums.
static int64_t embed_list(const ssd::EmbedPlan &p, int64_t rows) { return align256(rows * 8) * (p.tiles > 1 ? 2 : 1); }

size_t ssd_embedding_bwd_workspace_bytes(int64_t rows, int64_t vocab, int64_t dim) {
    if (check_embed(rows, vocab, dim) != SSD_OK) return (size_t)-1;
    const ssd::EmbedPlan p = ssd::embed_plan(rows, vocab, dim);
    return (size_t)(embed_list(p, rows) + align256(p.pieces * 2 * dim * 4));
}

ssd_status ssd_embedding_bwd(const void *dy, const int32_t *tokens, float scale, void *dtable, int accumulate, int64_t rows,
                             int64_t vocab, int64_t dim, ssd_dtype dy_dtype, ssd_dtype dtype, void *workspace,
                             size_t workspace_bytes, void *stream) {
    if (!dtable || (rows != 0 && (!dy || !tokens))) return SSD_ERR_NULL;
    if (!valid_dtype((int)dy_dtype) || !valid_dtype((int)dtype)) return SSD_ERR_UNSUPPORTED;
    ssd_status st = check_embed(rows, vocab, dim);
    if (st != SSD_OK) return st;
    if (misaligned((const char *)dy, (const char *)tokens, (const char *)dtable)) return SSD_ERR_ALIGN;
    if ((st = check_workspace((int64_t)ssd_embedding_bwd_workspace_bytes(rows, vocab, dim), workspace, workspace_bytes)) != SSD_OK) return st;
    if (any_overlap({{dtable, vocab * dim * esize(dtype)}}, {{dy, rows * dim * esize(dy_dtype)}, {tokens, rows * 4}})) return SSD_ERR_UNSUPPORTED;
    const ssd::EmbedPlan p = ssd::embed_plan(rows, vocab, dim);
    char *ws = static_cast<char *>(workspace);
    ssd::EmbedBwdArgs a = {};
    a.dy = dy; a.dtable = dtable; a.part = reinterpret_cast<float *>(ws + embed_list(p, rows)); a.rows = rows; a.vocab = (int)vocab;
    a.dim = (int)dim; a.accumulate = accumulate != 0; a.scale = scale;
    return ssd::launch_embed_bwd(a, p, tokens, reinterpret_cast<uint64_t *>(ws), reinterpret_cast<uint64_t *>(ws + align256(rows * 8)),
                                 dy_dtype, dtype, reinterpret_cast<hipStream_t>(stream));
}

ssd_status ssd_logits_process(const void *logits, void *out, const int32_t *tokens, int64_t capacity, const int32_t *lengths,
                              const int32_t *prompt, const float *repetition, const float *presence, const float *frequency,
                              const float *bias, int64_t bias_rows, const int32_t *mask, int64_t mask_rows, int64_t rows,
                              int64_t vocab, ssd_dtype dtype, void *stream) {
    if (rows != 0 && (!logits || !out)) return SSD_ERR_NULL;
    if (!tokens && (lengths || prompt || repetition || presence || frequency)) return SSD_ERR_NULL;
    if (!valid_dtype((int)dtype)) return SSD_ERR_UNSUPPORTED;
    if (rows < 0 || vocab <= 0 || (tokens && capacity < 0)) return SSD_ERR_SHAPE;
    if ((bias && bias_rows != 1 && bias_rows != rows) || (mask && mask_rows != 1 && mask_rows != rows)) return SSD_ERR_SHAPE;
    if (vocab > ((int64_t)1 << 28) || (tokens && capacity > INT32_MAX)) return SSD_ERR_UNSUPPORTED;
    if (rows > ssd::kMostThreads / 256 / ssd::logits_slices(vocab)) return SSD_ERR_UNSUPPORTED;
    if (misaligned((const char *)logits, (const char *)out, (const char *)tokens, (const char *)lengths, (const char *)prompt,
                   (const char *)repetition, (const char *)presence, (const char *)frequency, (const char *)bias, (const char *)mask))
        return SSD_ERR_ALIGN;
    if (rows == 0) return SSD_OK;
    const int64_t n = rows * vocab * esize(dtype), words = (vocab + 31) / 32;
    if (any_overlap({{out, n}}, {{logits == out ? nullptr : logits, n}, {tokens, rows * capacity * 4}, {lengths, rows * 4}, {prompt, rows * 4},
                                 {repetition, rows * 4}, {presence, rows * 4}, {frequency, rows * 4}, {bias, bias_rows * vocab * 4},
                                 {mask, mask_rows * words * 4}}))
        return SSD_ERR_UNSUPPORTED;
    ssd::LogitsArgs a = {};
    a.logits = logits; a.out = out; a.tokens = tokens; a.lengths = lengths; a.prompt = prompt; a.repetition = repetition;
    a.presence = presence; a.frequency = frequency; a.bias = bias; a.mask = reinterpret_cast<const uint32_t *>(mask);
    a.rows = rows; a.vocab = vocab; a.capacity = capacity; a.words = words; a.bias_rows = bias_rows; a.mask_rows = mask_rows;
    return ssd::launch_logits(a, dtype, reinterpret_cast<hipStream_t>(stream));
}

ssd_status ssd_int_quantize(const void *x, int8_t *q, float *scale, int64_t rows, int64_t dim, ssd_dtype dtype, void *stream) {
    if (rows != 0 && (!x || !q || !scale)) return SSD_ERR_NULL;
    if (!valid_dtype((int)dtype)) return SSD_ERR_UNSUPPORTED;
    if (rows < 0 || dim <= 0) return SSD_ERR_SHAPE;
    if (dim > kMostDim || rows > ((int64_t)1 << 41) / dim) return SSD_ERR_UNSUPPORTED;
    if (misaligned((const char *)x, (const char *)q, (const char *)scale)) return SSD_ERR_ALIGN;
    if (rows == 0) return SSD_OK;
    if (any_overlap({{q, rows * dim}, {scale, rows * 4}}, {{x, rows * dim * esize(dtype)}})) return SSD_ERR_UNSUPPORTED;
    return ssd::launch_int_quantize(x, q, scale, rows, dim, dtype, reinterpret_cast<hipStream_t>(stream));
}

static ssd_status check_int(int64_t rows, int64_t in, int64_t out) {
    if (rows < 0 || in <= 0 || out <= 0 || in % 16 != 0) return SSD_ERR_SHAPE;
    // 127 * 128 * 131072 < 2^31
    return rows > ((int64_t)1 << 24) || in > 131072 || out > kMostDim ? SSD_ERR_UNSUPPORTED : SSD_OK;
}

size_t ssd_linear_int_workspace_bytes(int64_t rows, int64_t in, int64_t out) {
    if (check_int(rows, in, out) != SSD_OK) return (size_t)-1;
    if (rows == 0) return 0;
    const ssd::LinearPlan p = ssd::linear_plan(rows, out, in, false, false);
    return p.splits > 1 ? (size_t)align256(p.splits * ssd::part_stride(rows, out) * 4) : 0;
}

ssd_status ssd_linear_int(const int8_t *xq, const float *xscale, const int8_t *wq, const float *wscale, const float *bias,
                         int act, const void *residual, void *y, int64_t rows, int64_t in, int64_t out, ssd_dtype dtype,
                         void *workspace, size_t workspace_bytes, void *stream) {
    if (rows != 0 && (!xq || !xscale || !wq || !wscale || !y)) return SSD_ERR_NULL;
    if (!valid_dtype((int)dtype) || act < SSD_ACT_NONE || act > SSD_ACT_GELU) return SSD_ERR_UNSUPPORTED;
    ssd_status st = check_int(rows, in, out);
    if (st != SSD_OK) return st;
    if (misaligned((const char *)xq, (const char *)xscale, (const char *)wq, (const char *)wscale, (const char *)bias,
                   (const char *)residual, (const char *)y))
        return SSD_ERR_ALIGN;
    if ((st = check_workspace((int64_t)ssd_linear_int_workspace_bytes(rows, in, out), workspace, workspace_bytes)) != SSD_OK) return st;
    if (rows == 0) return SSD_OK;
    const int64_t ny = rows * out * esize(dtype);
    if (any_overlap({{y, ny}}, {{xq, rows * in}, {xscale, rows * 4}, {wq, out * in}, {wscale, out * 4}, {bias, out * 4},
                                {y == residual ? nullptr : residual, ny}}))
        return SSD_ERR_UNSUPPORTED;
    ssd::LinearArgs a = {};
    a.x = xq; a.w = wq; a.xs = xscale; a.ws = wscale; a.bias = bias; a.res = residual; a.y = y; a.act = act;
    a.M = (int)rows; a.N = (int)out; a.ldx = a.ldw = in; a.kbytes = (uint32_t)in;
    a.part = static_cast<float *>(workspace);
    return ssd::launch_linear_int(a, ssd::linear_plan(rows, out, in, false, false), dtype, reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
