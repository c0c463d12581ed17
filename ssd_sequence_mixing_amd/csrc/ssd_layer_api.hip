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

__global__ void k_clear(float *p, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) p[i] = 0.f;
}

ssd_status clear(float *p, int64_t n, hipStream_t s) {
    if (n == 0) return SSD_OK;
    return ssd::launch(k_clear, dim3((unsigned)((n + 255) / 256)), dim3(256), s, p, n) == hipSuccess ? SSD_OK
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
    return align256(n * beams * 8) + align256(n * 8);
}

}  // namespace

extern "C" {

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
    if (rows == 0) return clear(dweight, dim, s);
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
    a.sums = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + align256(a.rows * a.lists * beams * 8));
    return ssd::launch_beam_select(a, batch, dtype, reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
