// Internal interface of the operators around the scan in a block: the two
// fused norms, the 8-bit checkpoints and the weight gradient that reads one.
// block_api.hip checks the arguments; the launchers take them as checked.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ssm.h"

namespace ssm {

// Widest normalised group (a workgroup of 1024 lanes holds 4 x 8 values each).
constexpr int64_t kNormMaxGroup = 32768;

inline int64_t ckpt8_width(int64_t width) { return (width + 31) / 32 * 32; }

struct NormShape {
    int64_t M;        // rows
    int W, G, Wg;     // width, groups, width of a group
    int io, res;      // ssm_dtype
    float eps, alpha; // alpha: residual scale
    bool after;       // gate after the norm
    int64_t ld_x, ld_z, ld_res, ld_out;
    int64_t scale_off;  // byte offset of a checkpoint's scale bytes
    int W32;
};

// Row slices of a backward: each is one row of per-column partial sums.
int norm_bwd_slices(const NormShape& s, bool gated);

struct GatedArgs {
    NormShape s;
    const void *y, *z;
    const float* w;
    void* out;
    float* rstd;
    uint8_t *y8, *z8, *out8;
};
int launch_norm_gated_fwd(const GatedArgs& a, hipStream_t stream);

struct GatedBwdArgs {
    NormShape s;
    const void *dout, *y, *z;
    const uint8_t *y8, *z8;
    const float *w, *rstd;
    void *d_y, *d_z;
    float* d_w;
    float* part;  // partial sums [slices][W]
};
int launch_norm_gated_bwd(const GatedBwdArgs& a, hipStream_t stream);

struct ResidualArgs {
    NormShape s;
    const void *b, *r;
    const float *w_post, *scale, *w;
    void *r_out, *h;
    float *rstd, *rstd_post;
    uint8_t *r8, *b8, *h8;
};
int launch_norm_residual_fwd(const ResidualArgs& a, hipStream_t stream);

struct ResidualBwdArgs {
    NormShape s;
    const void *dh, *dr_out, *r_out, *b;
    const uint8_t *r8, *b8;
    const float *w_post, *scale, *w, *rstd, *rstd_post;
    void *d_r, *d_b;
    float *d_w, *d_w_post, *d_scale;
    float* part;  // partial sums [2][slices][W]
};
int launch_norm_residual_bwd(const ResidualBwdArgs& a, hipStream_t stream);

// Sums S partial rows of W columns in a fixed order: d_w[c] = sum_s
// part[0][s][c] and, with T the same of part[1], d_w_post = alpha scale T and
// d_scale = alpha w_post T.  Null outputs are skipped, null factors are 1.
struct ColumnSums {
    float *d_w, *d_w_post = nullptr, *d_scale = nullptr;
    const float *scale = nullptr, *w_post = nullptr;
    float alpha = 1.0f;
};
int launch_column_sums(const float* part, int S, int W, const ColumnSums& out, hipStream_t stream);

int launch_ckpt8_pack(const void* x, int64_t ld, int64_t M, int64_t W, int dtype, uint8_t* out,
                      hipStream_t stream);
int launch_ckpt8_unpack(const uint8_t* x8, void* x, int64_t ld, int64_t M, int64_t W, int dtype,
                        hipStream_t stream);

size_t ckpt8_wgrad_workspace_bytes(int64_t M, int64_t W, int64_t O, int dtype);
int launch_ckpt8_wgrad(const void* dy, int64_t ld, const uint8_t* x8, float* dw, int64_t M, int64_t W,
                       int64_t O, int dtype, bool accumulate, void* ws, hipStream_t stream);

}  // namespace ssm
