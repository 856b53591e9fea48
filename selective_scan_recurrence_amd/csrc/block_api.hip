// The C ABI of the operators around the scan in a block (declared in
// include/ssm.h): argument checks on the host and dispatch to the launchers.
// Nothing here reads device memory or allocates.
#include <limits.h>
#include <math.h>

#include "block_internal.h"

namespace ssm {
namespace {

bool mul_ok(int64_t a, int64_t b, int64_t* out) { return !__builtin_mul_overflow(a, b, out); }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }  // NULL passes
bool known(int32_t dtype) { return dtype == SSM_F32 || dtype == SSM_BF16; }
size_t size_of(int32_t dtype) { return dtype == SSM_BF16 ? 2 : 4; }

// a row stride in elements: 0 is the dense width; rows * ld * 4 must fit
bool stride_ok(int64_t rows, int64_t width, int64_t* ld) {
    int64_t t;
    if (*ld == 0) *ld = width;
    return *ld >= width && mul_ok(rows, *ld, &t) && mul_ok(t, 8, &t);
}

int check_norm(const ssm_norm_desc* d, NormShape* out) {
    if (!d) return SSM_ERR_NULL;
    if (!known(d->io_dtype) || !known(d->res_dtype)) return SSM_ERR_DTYPE;
    if (d->reserved != 0 || (d->flags & ~(uint32_t)SSM_NORM_GATE_AFTER)) return SSM_ERR_SHAPE;
    if (d->n_rows < 0 || d->width < 1 || d->n_group < 1 || d->width > 1 << 22 ||
        d->n_group > d->width || d->width % d->n_group || d->width / d->n_group > kNormMaxGroup)
        return SSM_ERR_SHAPE;
    int64_t t;
    if (!mul_ok(d->n_rows, d->n_group, &t) || t > INT_MAX) return SSM_ERR_SHAPE;
    if (!(d->eps >= 0x1p-126f) || !isfinite(d->eps) || !isfinite(d->res_scale)) return SSM_ERR_SHAPE;
    NormShape s;
    s.M = d->n_rows; s.W = (int)d->width; s.G = (int)d->n_group; s.Wg = s.W / s.G;
    s.io = d->io_dtype; s.res = d->res_dtype; s.eps = d->eps; s.alpha = d->res_scale;
    s.after = d->flags & SSM_NORM_GATE_AFTER;
    s.ld_x = d->ld_x; s.ld_z = d->ld_z; s.ld_res = d->ld_res; s.ld_out = d->ld_out;
    if (!stride_ok(s.M, s.W, &s.ld_x) || !stride_ok(s.M, s.W, &s.ld_z) ||
        !stride_ok(s.M, s.W, &s.ld_res) || !stride_ok(s.M, s.W, &s.ld_out))
        return SSM_ERR_SHAPE;
    s.W32 = (int)ckpt8_width(s.W);
    s.scale_off = s.M * s.W32;
    *out = s;
    return SSM_OK;
}

// the residual norm has one group, and no f32 branch beside a bf16 stream
int check_residual(const ssm_norm_desc* d, NormShape* out) {
    const int rc = check_norm(d, out);
    if (rc) return rc;
    if (out->G != 1 || out->after) return SSM_ERR_SHAPE;
    return out->io == SSM_F32 && out->res == SSM_BF16 ? SSM_ERR_UNSUPPORTED : SSM_OK;
}

// partial rows of the gated norm's d_w, or of the residual norm's d_w and of its
// two sums over the branch: the larger, since a descriptor serves both
size_t norm_bwd_workspace(const NormShape& s) {
    const size_t gated = norm_bwd_slices(s, true), residual = s.G == 1 ? 2 * (size_t)norm_bwd_slices(s, false) : 0;
    const size_t n = (gated > residual ? gated : residual) * s.W * 4;
    return (n + 255) / 256 * 256;
}

// a checkpoint's dimensions
int check_ckpt(int64_t M, int64_t W) {
    int64_t t;
    if (M < 0 || W < 1 || W > INT_MAX - 1024 || !mul_ok(M, ckpt8_width(W), &t) || t > (int64_t)1 << 44)
        return SSM_ERR_SHAPE;
    return SSM_OK;
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" {

size_t ssm_ckpt8_bytes(int64_t n_rows, int64_t width, size_t* scale_offset) {
    if (check_ckpt(n_rows, width)) return 0;
    const size_t codes = (size_t)n_rows * (size_t)ckpt8_width(width);
    if (scale_offset) *scale_offset = codes;
    return codes + codes / 32;
}

int ssm_ckpt8_pack(const void* x, int64_t ld, int64_t n_rows, int64_t width, int32_t dtype,
                   void* ckpt, ssm_stream_t stream) {
    if (!known(dtype)) return SSM_ERR_DTYPE;
    if (check_ckpt(n_rows, width) || !stride_ok(n_rows, width, &ld)) return SSM_ERR_SHAPE;
    if (n_rows > 0 && (!x || !ckpt)) return SSM_ERR_NULL;
    if (!aligned(x, size_of(dtype)) || !aligned(ckpt, 16)) return SSM_ERR_ALIGN;
    return launch_ckpt8_pack(x, ld, n_rows, width, dtype, static_cast<uint8_t*>(ckpt),
                             static_cast<hipStream_t>(stream));
}

int ssm_ckpt8_unpack(const void* ckpt, void* x, int64_t ld, int64_t n_rows, int64_t width,
                     int32_t dtype, ssm_stream_t stream) {
    if (!known(dtype)) return SSM_ERR_DTYPE;
    if (check_ckpt(n_rows, width) || !stride_ok(n_rows, width, &ld)) return SSM_ERR_SHAPE;
    if (n_rows > 0 && (!x || !ckpt)) return SSM_ERR_NULL;
    if (!aligned(x, size_of(dtype)) || !aligned(ckpt, 16)) return SSM_ERR_ALIGN;
    return launch_ckpt8_unpack(static_cast<const uint8_t*>(ckpt), x, ld, n_rows, width, dtype,
                               static_cast<hipStream_t>(stream));
}

static int check_wgrad(int64_t n_rows, int64_t width, int64_t n_out, int32_t dtype) {
    int64_t t;
    if (!known(dtype)) return SSM_ERR_DTYPE;
    if (check_ckpt(n_rows, width) || n_rows > INT_MAX - 1024 || n_out < 1 || n_out > 1 << 22 ||
        width > 1 << 22 || !mul_ok(n_out, width, &t) || t > (int64_t)1 << 37)
        return SSM_ERR_SHAPE;
    return SSM_OK;
}

size_t ssm_ckpt8_wgrad_workspace_bytes(int64_t n_rows, int64_t width, int64_t n_out, int32_t dtype) {
    if (check_wgrad(n_rows, width, n_out, dtype)) return 0;
    return (ckpt8_wgrad_workspace_bytes(n_rows, width, n_out, dtype) + 255) / 256 * 256;
}

int ssm_ckpt8_wgrad(const void* dy, int64_t ld, const void* ckpt, float* dw, int64_t n_rows,
                    int64_t width, int64_t n_out, int32_t dtype, int32_t accumulate,
                    void* workspace, size_t workspace_bytes, ssm_stream_t stream) {
    const int rc = check_wgrad(n_rows, width, n_out, dtype);
    if (rc) return rc;
    if (!stride_ok(n_rows, n_out, &ld) || ld > 1 << 22) return SSM_ERR_SHAPE;
    const size_t need = ssm_ckpt8_wgrad_workspace_bytes(n_rows, width, n_out, dtype);
    if (!dw || (n_rows > 0 && (!dy || !ckpt)) || (need && !workspace)) return SSM_ERR_NULL;
    if (workspace_bytes < need) return SSM_ERR_WORKSPACE;
    if (!aligned(dy, size_of(dtype)) || !aligned(ckpt, 16) || !aligned(dw, 4) || !aligned(workspace, 256))
        return SSM_ERR_ALIGN;
    return launch_ckpt8_wgrad(dy, ld, static_cast<const uint8_t*>(ckpt), dw, n_rows, width, n_out, dtype,
                              accumulate != 0, workspace, static_cast<hipStream_t>(stream));
}

size_t ssm_norm_bwd_workspace_bytes(const ssm_norm_desc* desc) {
    NormShape s;
    return check_norm(desc, &s) == SSM_OK ? norm_bwd_workspace(s) : 0;
}

int ssm_norm_gated_fwd(const ssm_norm_desc* desc, const void* y, const void* z, const float* w,
                       void* out, float* rstd, void* y8, void* z8, void* out8, ssm_stream_t stream) {
    NormShape s;
    const int rc = check_norm(desc, &s);
    if (rc) return rc;
    // a checkpoint's blocks may not straddle two groups
    if ((y8 || z8 || out8) && s.G > 1 && s.Wg % 32) return SSM_ERR_UNSUPPORTED;
    if (!w || (s.M > 0 && (!y || !out)) || (z8 && !z)) return SSM_ERR_NULL;
    const size_t es = size_of(s.io);
    if (!aligned(y, es) || !aligned(z, es) || !aligned(out, es) || !aligned(w, 4) || !aligned(rstd, 4) ||
        !aligned(y8, 16) || !aligned(z8, 16) || !aligned(out8, 16))
        return SSM_ERR_ALIGN;
    GatedArgs a = {s, y, z, w, out, rstd, static_cast<uint8_t*>(y8), static_cast<uint8_t*>(z8),
                   static_cast<uint8_t*>(out8)};
    return launch_norm_gated_fwd(a, static_cast<hipStream_t>(stream));
}

int ssm_norm_gated_bwd(const ssm_norm_desc* desc, const void* dout, const void* y, const void* z,
                       const void* y8, const void* z8, const float* w, const float* rstd, void* d_y,
                       void* d_z, float* d_w, void* workspace, size_t workspace_bytes,
                       ssm_stream_t stream) {
    NormShape s;
    const int rc = check_norm(desc, &s);
    if (rc) return rc;
    if ((y8 || z8) && s.G > 1 && s.Wg % 32) return SSM_ERR_UNSUPPORTED;
    // y as a tensor or as its checkpoint, not both; the same for z
    if ((y && y8) || (z && z8)) return SSM_ERR_UNSUPPORTED;
    if (!w || (s.M > 0 && (!dout || !rstd || !(y || y8))) || (d_z && !(z || z8)) || (d_w && !workspace))
        return SSM_ERR_NULL;
    if (d_w && workspace_bytes < norm_bwd_workspace(s)) return SSM_ERR_WORKSPACE;
    const size_t es = size_of(s.io);
    if (!aligned(dout, es) || !aligned(y, es) || !aligned(z, es) || !aligned(d_y, es) || !aligned(d_z, es) ||
        !aligned(y8, 16) || !aligned(z8, 16) || !aligned(w, 4) || !aligned(rstd, 4) || !aligned(d_w, 4) ||
        !aligned(workspace, 256))
        return SSM_ERR_ALIGN;
    GatedBwdArgs a = {s, dout, y, z, static_cast<const uint8_t*>(y8), static_cast<const uint8_t*>(z8),
                      w, rstd, d_y, d_z, d_w, static_cast<float*>(workspace)};
    return launch_norm_gated_bwd(a, static_cast<hipStream_t>(stream));
}

int ssm_norm_residual_fwd(const ssm_norm_desc* desc, const void* b, const void* r, const float* w_post,
                          const float* scale, const float* w, void* r_out, void* h, float* rstd,
                          float* rstd_post, void* r8, void* b8, void* h8, ssm_stream_t stream) {
    NormShape s;
    const int rc = check_residual(desc, &s);
    if (rc) return rc;
    if (!w || (s.M > 0 && ((!b && !r) || !h)) || (!b && (w_post || scale || b8) && s.M > 0) ||
        (rstd_post && !w_post))
        return SSM_ERR_NULL;
    const size_t es = size_of(s.io), rs = size_of(s.res);
    if (!aligned(b, es) || !aligned(r, rs) || !aligned(w_post, 4) || !aligned(scale, 4) || !aligned(w, 4) ||
        !aligned(r_out, rs) || !aligned(h, es) || !aligned(rstd, 4) || !aligned(rstd_post, 4) ||
        !aligned(r8, 16) || !aligned(b8, 16) || !aligned(h8, 16))
        return SSM_ERR_ALIGN;
    ResidualArgs a = {s, b, r, w_post, scale, w, r_out, h, rstd, rstd_post, static_cast<uint8_t*>(r8),
                      static_cast<uint8_t*>(b8), static_cast<uint8_t*>(h8)};
    return launch_norm_residual_fwd(a, static_cast<hipStream_t>(stream));
}

int ssm_norm_residual_bwd(const ssm_norm_desc* desc, const void* dh, const void* dr_out, const void* r_out,
                          const void* r8, const void* b, const void* b8, const float* w_post,
                          const float* scale, const float* w, const float* rstd, const float* rstd_post,
                          void* d_r, void* d_b, float* d_w, float* d_w_post, float* d_scale,
                          void* workspace, size_t workspace_bytes, ssm_stream_t stream) {
    NormShape s;
    const int rc = check_residual(desc, &s);
    if (rc) return rc;
    if ((r_out && r8) || (b && b8)) return SSM_ERR_UNSUPPORTED;
    const bool sums = d_w || d_w_post || d_scale;
    if (!w || (d_w_post && !w_post) || (sums && !workspace) ||
        (s.M > 0 && (!dh || !rstd || !(r_out || r8) || ((w_post || d_scale) && !(b || b8)) ||
                     (w_post && !rstd_post))))
        return SSM_ERR_NULL;
    if (sums && workspace_bytes < norm_bwd_workspace(s)) return SSM_ERR_WORKSPACE;
    const size_t es = size_of(s.io), rs = size_of(s.res);
    if (!aligned(dh, es) || !aligned(dr_out, rs) || !aligned(r_out, rs) || !aligned(r8, 16) ||
        !aligned(b, es) || !aligned(b8, 16) || !aligned(w_post, 4) || !aligned(scale, 4) || !aligned(w, 4) ||
        !aligned(rstd, 4) || !aligned(rstd_post, 4) || !aligned(d_r, rs) || !aligned(d_b, es) ||
        !aligned(d_w, 4) || !aligned(d_w_post, 4) || !aligned(d_scale, 4) || !aligned(workspace, 256))
        return SSM_ERR_ALIGN;
    ResidualBwdArgs a = {s, dh, dr_out, r_out, b, static_cast<const uint8_t*>(r8),
                         static_cast<const uint8_t*>(b8), w_post, scale, w, rstd, rstd_post, d_r, d_b,
                         d_w, d_w_post, d_scale, static_cast<float*>(workspace)};
    return launch_norm_residual_bwd(a, static_cast<hipStream_t>(stream));
}

}  // extern "C"
