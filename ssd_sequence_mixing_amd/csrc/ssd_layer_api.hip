// C ABI of libssd, continued: the operators around the core in a decoder
// (norm, projections, beam search). Every check runs on the host before
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

__global__ void k_clear(uint16_t *p, int64_t n) {
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) p[i] = 0;
}

// Zeros over an even number of bytes (weights of any size: 2^33 values are more threads than a launch takes).
ssd_status clear(void *p, int64_t bytes, hipStream_t s) {
    if (!p || bytes == 0) return SSD_OK;
    const int64_t n = bytes / 2, blocks = (n + 255) / 256, most = 1 << 16;
    return ssd::launch(k_clear, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), s,
                       static_cast<uint16_t *>(p), n) == hipSuccess
               ? SSD_OK
               : SSD_ERR_HIP;
}

ssd_status check_workspace(int64_t need, const void *workspace, size_t workspace_bytes) {
    if (need == 0) return SSD_OK;
    if (!workspace || workspace_bytes < (size_t)need) return SSD_ERR_WORKSPACE;
    return ((uintptr_t)workspace & 255u) ? SSD_ERR_ALIGN : SSD_OK;
}

// Shapes and types of the norm family. mx: blocks of 32 may not cross a group.
ssd_status check_norm(int64_t rows, int64_t dim, int64_t groups, int dtype, int residual_dtype, bool mx) {
    if (!valid_dtype(dtype) || !valid_dtype(residual_dtype)) return SSD_ERR_UNSUPPORTED;
    if (dtype == SSD_F32 && residual_dtype == SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (rows < 0 || dim <= 0 || groups <= 0 || dim % groups != 0) return SSD_ERR_SHAPE;
    const int64_t n = dim / groups;
    if (mx && n % 32 != 0) return SSD_ERR_SHAPE;
    if (n > 65536 || groups > 65535 || rows > (int64_t)INT32_MAX / groups) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

ssd_status norm_impl(const void *x, const void *residual, const float *weight, float eps, void *residual_out,
                     void *y, uint8_t *q, uint8_t *scale, float *rstd, int64_t rows, int64_t dim, int64_t groups,
                     ssd_dtype dtype, ssd_dtype residual_dtype, bool mx, void *stream) {
    if (rows != 0 && (!x || !weight || (mx ? !q || !scale : !y))) return SSD_ERR_NULL;
    if (rows != 0 && (!residual != !residual_out)) return SSD_ERR_NULL;
    const ssd_status st = check_norm(rows, dim, groups, (int)dtype, (int)residual_dtype, mx);
    if (st != SSD_OK) return st;
    if (misaligned((const char *)x, (const char *)residual, (const char *)weight, (const char *)residual_out,
                   (const char *)y, (const char *)q, (const char *)scale, (const char *)rstd))
        return SSD_ERR_ALIGN;
    if (rows == 0) return SSD_OK;
    ssd::NormArgs a = {};
    a.x = x; a.res = residual; a.w = weight; a.res_out = residual_out; a.y = y; a.q = q; a.scale = scale;
    a.rstd = rstd; a.rows = rows * groups; a.groups = groups; a.Dg = (int)(dim / groups); a.eps = eps;
    a.dtype = dtype; a.res_dtype = residual_dtype;
    return ssd::launch_rms_norm(a, reinterpret_cast<hipStream_t>(stream));
}

// Bytes of a selection's workspace, or -1.
int64_t beam_bytes(int64_t batch, int64_t beams, int64_t vocab, int *lists, int *tiles, ssd_status *why) {
    *why = SSD_ERR_SHAPE;
    if (batch < 0 || beams <= 0 || vocab <= 0) return -1;
    *why = SSD_ERR_UNSUPPORTED;
    // 16 beams: a wavefront sorts 64 keys, the list and up to 48 new ones
    if (beams > 16 || vocab > ((int64_t)1 << 28) || batch > (int64_t)INT32_MAX / 16 / 64) return -1;
    *why = SSD_OK;
    ssd::beam_plan(vocab, lists, tiles);
    const int64_t n = batch * beams * *lists;
    *why = SSD_ERR_UNSUPPORTED;
    if (n > ssd::kMostThreads / 256 * 4) return -1;  // a wavefront for each, 4 to a work-group: 137 GB of logits and more
    *why = SSD_OK;
    return align256(n * beams * 8) + align256(n * 8);
}

constexpr int64_t kMostDim = (int64_t)1 << 20;   // in and out: 256 rows stay under 2 GiB
constexpr int64_t kMostRows = (int64_t)1 << 24;

ssd_status check_linear(int64_t rows, int64_t in, int64_t out, int act, int64_t most_rows) {
    if (act < SSD_ACT_NONE || act > SSD_ACT_GELU) return SSD_ERR_UNSUPPORTED;
    if (rows < 0 || in <= 0 || out <= 0) return SSD_ERR_SHAPE;
    if (rows > most_rows || in > kMostDim || out > kMostDim) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

int64_t align16(int64_t v) { return (v + 15) & ~(int64_t)15; }

// A product's operands are read while it writes: whether an output lies on one. Bytes of each behind its address.
struct Span {
    const void *p;
    int64_t bytes;
};
template <size_t O, size_t I>
bool any_overlap(const Span (&out)[O], const Span (&in)[I]) {
    for (const Span &o : out)
        for (const Span &i : in)
            if (ssd::overlap(o.p, o.bytes, i.p, i.bytes)) return true;
    return false;
}

// Workspace of a product: copies of the operands, in rows of multiples of 16 bytes, where
// theirs begin at odd multiples of 2 (and there are more than a few), and the parts of a split sum.
struct LinearLayout {
    ssd::LinearPlan plan;
    int64_t ld, xpad, wpad, xs, ws, part, total;
};
LinearLayout linear_layout(int64_t rows, int64_t in, int64_t out, ssd_dtype dtype) {
    LinearLayout l = {};
    if (rows == 0) return l;
    const int64_t bytes = in * esize(dtype);
    l.ld = align16(bytes);
    l.plan = ssd::linear_plan(rows, out, l.ld, dtype == SSD_F32, false);
    if (!l.plan.bm || bytes % 4 == 0) {  // operands as they are
        l.ld = bytes;
    } else if (l.ld != bytes) {
        l.xpad = align256(rows * l.ld);
        l.wpad = align256(out * l.ld);
    }
    if (l.plan.splits > 1) l.part = align256(l.plan.splits * ssd::part_stride(rows, out) * 4);
    l.total = l.xpad + l.wpad + l.part;
    return l;
}
// 8-bit operands: the tile kernel takes a step's 4 scales of a row as one word.
LinearLayout linear_mx_layout(int64_t rows, int64_t in, int64_t out) {
    LinearLayout l = {};
    if (rows == 0) return l;
    l.plan = ssd::linear_plan(rows, out, in, false, false);
    l.ld = in / 32;
    if (l.plan.bm && l.ld % 4 != 0) {
        l.ld = (l.ld + 3) & ~(int64_t)3;
        l.xs = align256(rows * l.ld);
        l.ws = align256(out * l.ld);
    }
    if (l.plan.splits > 1) l.part = align256(l.plan.splits * ssd::part_stride(rows, out) * 4);
    l.total = l.xs + l.ws + l.part;
    return l;
}

// Workspace of the gradients, one after the other: dz (where it is not dy
// itself); bf16: copies of w and x with rows of 16-byte multiples, where theirs are
// not; fp32: dz, w and x transposed (rows of ldt / ldz values); the shares of
// dbias, of dbrows rows each; the parts of the two products' sums.
struct LinearBwdLayout {
    ssd::LinearPlan px, pw;
    int64_t ldz, ldt, ldk, kz, dbrows, dz, dzt, w, x, db, part, total;  // kz: bytes of dz along its row that a product takes
};
LinearBwdLayout linear_bwd_layout(int64_t rows, int64_t in, int64_t out, int act, bool want_dx, bool want_dw,
                                  bool want_db, ssd_dtype dtype) {
    LinearBwdLayout l = {};
    if (rows == 0) return l;
    const int64_t es = esize(dtype);
    const bool bf = dtype == SSD_BF16;
    l.ldz = align16(out * es) / es;
    l.ldt = align16(rows * es) / es;
    l.ldk = align16(in * es) / es;
    l.kz = l.ldz * es;
    if ((want_dx || want_dw) && (act != SSD_ACT_NONE || l.ldz != out)) {
        // its own rows begin at whole cache lines: 128 bytes of a row are then one line, not two
        // (out = 3352: dx 94 us without, 84 with, on a cool GPU)
        l.ldz = (out * es + 127) / 128 * 128 / es;
        l.dz = align256(rows * l.ldz * es);
    }
    int64_t px = 0, pw = 0;
    if (want_dx) {
        l.w = bf ? (l.ldk != in ? align256(out * l.ldk * es) : 0) : align256(in * l.ldz * es);
        l.px = ssd::linear_plan(rows, in, l.kz, !bf, bf);
        if (l.px.splits > 1) px = align256(l.px.splits * ssd::part_stride(rows, in) * 4);
    }
    if (want_dw) {
        l.x = bf ? (l.ldk != in ? align256(rows * l.ldk * es) : 0) : align256(in * l.ldt * es);
        if (!bf) l.dzt = align256(l.ldz * l.ldt * es);
        l.pw = ssd::linear_plan(out, in, l.ldt * es, !bf, bf);
        if (l.pw.splits > 1) pw = align256(l.pw.splits * ssd::part_stride(out, in) * 4);
    }
    l.dbrows = ssd::dz_rows(rows, l.ldz);
    if (want_db) l.db = align256((rows + l.dbrows - 1) / l.dbrows * out * 4);
    l.part = px > pw ? px : pw;
    l.total = l.dz + l.dzt + l.w + l.x + l.db + l.part;
    return l;
}

}  // namespace

extern "C" {

size_t ssd_linear_workspace_bytes(int64_t rows, int64_t in, int64_t out, ssd_dtype dtype) {
    if (!valid_dtype((int)dtype) || check_linear(rows, in, out, SSD_ACT_NONE, kMostRows) != SSD_OK) return (size_t)-1;
    return (size_t)linear_layout(rows, in, out, dtype).total;
}

ssd_status ssd_linear(const void *x, const void *w, const float *bias, int act, const void *residual, void *y,
                      void *preact, int64_t rows, int64_t in, int64_t out, ssd_dtype dtype, void *workspace,
                      size_t workspace_bytes, void *stream) {
    if (rows != 0 && (!x || !w || !y)) return SSD_ERR_NULL;
    if (!valid_dtype((int)dtype)) return SSD_ERR_UNSUPPORTED;
    ssd_status st = check_linear(rows, in, out, act, kMostRows);
    if (st != SSD_OK) return st;
    if (misaligned((const char *)x, (const char *)w, (const char *)bias, (const char *)residual, (const char *)y,
                   (const char *)preact))
        return SSD_ERR_ALIGN;
    const LinearLayout l = linear_layout(rows, in, out, dtype);
    if ((st = check_workspace(l.total, workspace, workspace_bytes)) != SSD_OK) return st;
    if (rows == 0) return SSD_OK;
    const int64_t es = esize(dtype), ny = rows * out * es;
    if (any_overlap({{y, ny}, {preact, ny}}, {{x, rows * in * es}, {w, out * in * es}, {bias, out * 4}}) ||
        (y != residual && ssd::overlap(y, ny, residual, ny)) || ssd::overlap(preact, ny, residual, ny))
        return SSD_ERR_UNSUPPORTED;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    ssd::LinearArgs a = {};
    a.x = x; a.w = w; a.bias = bias; a.res = residual; a.y = y; a.pre = preact; a.act = act;
    a.M = (int)rows; a.N = (int)out; a.ldx = a.ldw = l.ld; a.kbytes = (uint32_t)l.ld;
    if (l.xpad) {
        st = ssd::launch_pad(x, ws, rows, w, ws + l.xpad, out, in, l.ld / es, (int)es, s);
        if (st != SSD_OK) return st;
        a.x = ws;
        a.w = ws + l.xpad;
    }
    a.part = reinterpret_cast<float *>(ws + l.xpad + l.wpad);
    return ssd::launch_linear(a, l.plan, false, dtype, s);
}

size_t ssd_linear_mx_workspace_bytes(int64_t rows, int64_t in, int64_t out) {
    if (check_linear(rows, in, out, SSD_ACT_NONE, kMostRows) != SSD_OK || in % 32 != 0) return (size_t)-1;
    return (size_t)linear_mx_layout(rows, in, out).total;
}

ssd_status ssd_linear_mx(const uint8_t *xq, const uint8_t *xscale, const uint8_t *wq, const uint8_t *wscale,
                         const float *bias, int act, const void *residual, void *y, int64_t rows, int64_t in,
                         int64_t out, void *workspace, size_t workspace_bytes, void *stream) {
    if (rows != 0 && (!xq || !xscale || !wq || !wscale || !y)) return SSD_ERR_NULL;
    ssd_status st = check_linear(rows, in, out, act, kMostRows);
    if (st != SSD_OK) return st;
    if (in % 32 != 0) return SSD_ERR_SHAPE;
    if (misaligned((const char *)xq, (const char *)xscale, (const char *)wq, (const char *)wscale,
                   (const char *)bias, (const char *)residual, (const char *)y))
        return SSD_ERR_ALIGN;
    const LinearLayout l = linear_mx_layout(rows, in, out);
    if ((st = check_workspace(l.total, workspace, workspace_bytes)) != SSD_OK) return st;
    if (rows == 0) return SSD_OK;
    const int64_t ny = rows * out * 2;
    if (any_overlap({{y, ny}}, {{xq, rows * in}, {xscale, rows * in / 32}, {wq, out * in}, {wscale, out * in / 32}, {bias, out * 4}}) ||
        (y != residual && ssd::overlap(y, ny, residual, ny)))
        return SSD_ERR_UNSUPPORTED;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    ssd::LinearArgs a = {};
    a.x = xq; a.w = wq; a.xscale = xscale; a.wscale = wscale; a.bias = bias; a.res = residual; a.y = y; a.act = act;
    a.M = (int)rows; a.N = (int)out; a.ldx = a.ldw = in; a.lds = l.ld; a.kbytes = (uint32_t)in;
    if (l.xs) {
        st = ssd::launch_pad(xscale, ws, rows, wscale, ws + l.xs, out, in / 32, l.ld, 1, s);
        if (st != SSD_OK) return st;
        a.xscale = reinterpret_cast<uint8_t *>(ws);
        a.wscale = reinterpret_cast<uint8_t *>(ws + l.xs);
    }
    a.part = reinterpret_cast<float *>(ws + l.xs + l.ws);
    return ssd::launch_linear(a, l.plan, true, SSD_BF16, s);
}

size_t ssd_linear_bwd_workspace_bytes(int64_t rows, int64_t in, int64_t out, int act, ssd_dtype dtype) {
    if (!valid_dtype((int)dtype) || check_linear(rows, in, out, act, kMostDim) != SSD_OK) return (size_t)-1;
    return (size_t)linear_bwd_layout(rows, in, out, act, true, true, true, dtype).total;
}

ssd_status ssd_linear_bwd(const void *dy, const void *x, const void *w, int act, const void *preact, void *dx,
                          void *dw, float *dbias, int64_t rows, int64_t in, int64_t out, ssd_dtype dtype,
                          void *workspace, size_t workspace_bytes, void *stream) {
    if (rows != 0 && (!dy || (dx && !w) || (dw && !x) || (act != SSD_ACT_NONE && !preact))) return SSD_ERR_NULL;
    if (!valid_dtype((int)dtype)) return SSD_ERR_UNSUPPORTED;
    ssd_status st = check_linear(rows, in, out, act, kMostDim);
    if (st != SSD_OK) return st;
    if (misaligned((const char *)dy, (const char *)x, (const char *)w, (const char *)preact, (const char *)dx,
                   (const char *)dw, (const char *)dbias))
        return SSD_ERR_ALIGN;
    const LinearBwdLayout l = linear_bwd_layout(rows, in, out, act, dx, dw, dbias, dtype);
    if ((st = check_workspace(l.total, workspace, workspace_bytes)) != SSD_OK) return st;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const int64_t es = esize(dtype);
    if (rows == 0) {
        if ((st = clear(dw, out * in * es, s)) != SSD_OK) return st;
        return clear(dbias, out * 4, s);
    }
    const int64_t ny = rows * out * es, nx = rows * in * es, nw = out * in * es;
    if (any_overlap({{dx, nx}, {dw, nw}, {dbias, out * 4}},
                    {{dy, ny}, {dw ? x : nullptr, nx}, {dx ? w : nullptr, nw}, {act != SSD_ACT_NONE ? preact : nullptr, ny}}))
        return SSD_ERR_UNSUPPORTED;
    char *ws = static_cast<char *>(workspace);
    char *dz = ws, *dzt = dz + l.dz, *wc = dzt + l.dzt, *xc = wc + l.w;
    float *db = reinterpret_cast<float *>(xc + l.x), *part = reinterpret_cast<float *>(xc + l.x + l.db);
    const bool bf = dtype == SSD_BF16;
    if (l.dz || l.db) {
        st = ssd::launch_dz(dy, preact, act, l.dz ? dz : nullptr, l.db ? db : nullptr, rows, out, l.ldz, dtype, s);
        if (st != SSD_OK) return st;
    }
    if (dbias && (st = ssd::launch_column_sums(db, dbias, (int)((rows + l.dbrows - 1) / l.dbrows), out, s)) != SSD_OK) return st;
    const void *z = l.dz ? dz : dy;
    if (dx) {
        ssd::LinearArgs a = {};
        a.x = z; a.y = dx; a.part = part; a.M = (int)rows; a.N = (int)in; a.ldx = l.ldz * es; a.kbytes = (uint32_t)l.kz;
        a.w = w;
        if (l.w) {
            st = bf ? ssd::launch_pad(w, wc, out, w, wc, 0, in, l.ldk, 2, s) : ssd::launch_transpose(w, wc, out, in, l.ldz, s);
            if (st != SSD_OK) return st;
            a.w = wc;
        }
        a.ldw = bf ? l.ldk * es : a.ldx;
        a.wt = bf;
        a.krows = (int)out;
        if ((st = ssd::launch_linear(a, l.px, false, dtype, s)) != SSD_OK) return st;
    }
    if (dw) {
        ssd::LinearArgs a = {};
        a.y = dw; a.part = part; a.M = (int)out; a.N = (int)in; a.kbytes = (uint32_t)(l.ldt * es);
        a.x = z; a.w = x;
        if (l.x) {
            st = bf ? ssd::launch_pad(x, xc, rows, x, xc, 0, in, l.ldk, 2, s) : ssd::launch_transpose(x, xc, rows, in, l.ldt, s);
            if (st != SSD_OK) return st;
            a.w = xc;
        }
        if (bf) {
            a.ldx = l.ldz * es; a.ldw = l.ldk * es; a.xt = a.wt = true; a.krows = (int)rows;
        } else {
            // z has rows of ldz values, and only `out` of them are rows of the transpose
            if ((st = ssd::launch_transpose(z, dzt, rows, l.dz ? l.ldz : out, l.ldt, s)) != SSD_OK) return st;
            a.x = dzt; a.ldx = a.ldw = l.ldt * es;
        }
        if ((st = ssd::launch_linear(a, l.pw, false, dtype, s)) != SSD_OK) return st;
    }
    return SSD_OK;
}

ssd_status ssd_rms_norm(const void *x, const void *residual, const float *weight, float eps, void *residual_out,
                        void *y, float *rstd, int64_t rows, int64_t dim, int64_t groups, ssd_dtype dtype,
                        ssd_dtype residual_dtype, void *stream) {
    return norm_impl(x, residual, weight, eps, residual_out, y, nullptr, nullptr, rstd, rows, dim, groups, dtype,
                     residual_dtype, false, stream);
}

ssd_status ssd_rms_norm_mx(const void *x, const void *residual, const float *weight, float eps, void *residual_out,
                           uint8_t *q, uint8_t *scale, int64_t rows, int64_t dim, int64_t groups, ssd_dtype dtype,
                           ssd_dtype residual_dtype, void *stream) {
    return norm_impl(x, residual, weight, eps, residual_out, nullptr, q, scale, nullptr, rows, dim, groups, dtype,
                     residual_dtype, true, stream);
}

ssd_status ssd_mx_quantize(const void *x, uint8_t *q, uint8_t *scale, int64_t rows, int64_t dim, ssd_dtype dtype,
                           void *stream) {
    if (rows != 0 && (!x || !q || !scale)) return SSD_ERR_NULL;
    if (!valid_dtype((int)dtype)) return SSD_ERR_UNSUPPORTED;
    if (rows < 0 || dim <= 0 || dim % 32 != 0) return SSD_ERR_SHAPE;
    if (rows > ((int64_t)1 << 41) / dim) return SSD_ERR_UNSUPPORTED;
    if (misaligned((const char *)x, (const char *)q, (const char *)scale)) return SSD_ERR_ALIGN;
    if (rows == 0) return SSD_OK;
    return ssd::launch_mx_quantize(x, q, scale, rows * dim, dtype, reinterpret_cast<hipStream_t>(stream));
}

size_t ssd_rms_norm_bwd_workspace_bytes(int64_t rows, int64_t dim, int64_t groups, ssd_dtype dtype,
                                        ssd_dtype residual_dtype) {
    if (check_norm(rows, dim, groups, (int)dtype, (int)residual_dtype, false) != SSD_OK) return (size_t)-1;
    if (rows == 0) return 0;
    return (size_t)align256((int64_t)ssd::norm_bwd_blocks(rows, groups, dim / groups) * dim * 4);
}

ssd_status ssd_rms_norm_bwd(const void *dy, const void *h, const float *weight, const float *rstd,
                            const void *d_residual_out, void *dx, void *d_residual, float *dweight, int64_t rows,
                            int64_t dim, int64_t groups, ssd_dtype dtype, ssd_dtype residual_dtype, void *workspace,
                            size_t workspace_bytes, void *stream) {
    if (!dweight || (rows != 0 && (!dy || !h || !weight || !rstd || !dx))) return SSD_ERR_NULL;
    ssd_status st = check_norm(rows, dim, groups, (int)dtype, (int)residual_dtype, false);
    if (st != SSD_OK) return st;
    if (d_residual && dtype == residual_dtype) return SSD_ERR_UNSUPPORTED;  // dx is it
    if (misaligned((const char *)dy, (const char *)h, (const char *)weight, (const char *)rstd,
                   (const char *)d_residual_out, (const char *)dx, (const char *)d_residual, (const char *)dweight))
        return SSD_ERR_ALIGN;
    const int64_t need = (int64_t)ssd_rms_norm_bwd_workspace_bytes(rows, dim, groups, dtype, residual_dtype);
    if ((st = check_workspace(need, workspace, workspace_bytes)) != SSD_OK) return st;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (rows == 0) return clear(dweight, dim * 4, s);
    ssd::NormBwdArgs a = {};
    a.dy = dy; a.h = h; a.dres = d_residual_out; a.w = weight; a.rstd = rstd; a.dx = dx; a.dh = d_residual;
    a.dw = dweight; a.part = static_cast<float *>(workspace); a.rows = rows; a.groups = groups;
    a.Dg = (int)(dim / groups); a.nb = ssd::norm_bwd_blocks(rows, groups, dim / groups);
    a.dtype = dtype; a.res_dtype = residual_dtype;
    return ssd::launch_rms_norm_bwd(a, s);
}

size_t ssd_beam_select_workspace_bytes(int64_t batch, int64_t beams, int64_t vocab) {
    int lists, tiles;
    ssd_status why;
    return (size_t)beam_bytes(batch, beams, vocab, &lists, &tiles, &why);
}

ssd_status ssd_beam_select(const void *logits, const float *scores, const uint8_t *finished, int64_t eos,
                           float *next_scores, int32_t *parent, int32_t *token, uint8_t *next_finished,
                           int64_t batch, int64_t beams, int64_t vocab, ssd_dtype dtype, void *workspace,
                           size_t workspace_bytes, void *stream) {
    if (batch != 0 && (!logits || !scores || !next_scores || !parent || !token)) return SSD_ERR_NULL;
    if (!valid_dtype((int)dtype)) return SSD_ERR_UNSUPPORTED;
    ssd::BeamArgs a = {};
    ssd_status st;
    const int64_t need = beam_bytes(batch, beams, vocab, &a.lists, &a.tiles, &st);
    if (need < 0) return st;
    if (eos < -1 || eos >= vocab || (finished && eos < 0)) return SSD_ERR_SHAPE;
    if (misaligned((const char *)logits, (const char *)scores, (const char *)finished, (const char *)next_scores,
                   (const char *)parent, (const char *)token, (const char *)next_finished))
        return SSD_ERR_ALIGN;
    if ((st = check_workspace(need, workspace, workspace_bytes)) != SSD_OK) return st;
    if (batch == 0) return SSD_OK;
    a.logits = logits; a.scores = scores; a.finished = finished; a.out_scores = next_scores; a.parent = parent;
    a.token = token; a.out_finished = next_finished; a.rows = batch * beams; a.beams = (int)beams; a.V = (int)vocab;
    a.eos = (int)eos;
    a.keys = static_cast<uint64_t *>(workspace);
    a.sums = reinterpret_cast<double *>(static_cast<char *>(workspace) + align256(a.rows * a.lists * beams * 8));
    return ssd::launch_beam_select(a, batch, dtype, reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
