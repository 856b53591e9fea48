// The norm between two blocks, forward and backward.  Per row, with v = b (or,
// with a norm after the block, v = b rstd_post) and the column constants
// e = alpha scale w_post (factors that are not given are 1):
//   r' = r + e v                     (residual add and scale)
//   h  = r' rstd w                   (norm before the next block)
// with rstd = 1 / sqrt(mean r'^2 + eps), rstd_post the same of b; and, with
// c() the mean over the row:
//   x  = r' rstd, dn = dh w, dx = rstd (dn - x c(dn x)) + d_r_out,  d_r = dx
//   dm = e dx;  d_b = dm,  or  rstd_post (dm - v c(dm v))
//   d_w = sum_rows dh x;  S = sum_rows dx v:
//   d_w_post = alpha scale S,  d_scale = alpha w_post S
// All of it in f32; what is stored in fewer bits is rounded once.
//
// Bound by HBM: each input is read once and each output written once, the row
// held in registers between its sums and the outputs (norm_rows.h).
#include "norm_residual.h"

namespace ssm {
namespace {

struct FwdP {
    const void *b, *r;
    const float *w_post, *scale, *w;
    void *r_out, *h;
    float *rstd, *rstd_post;
    uint8_t *r8, *b8, *h8;
    int64_t ld_x, ld_res, ld_out, M, scale_off;
    int W, W32, slices;
    float eps, inv_n, alpha;
};

// Workgroup i takes every slices-th row (or set of rows) from i on, and loads
// the next one while it works on the present one.
template <typename T, typename R, typename RS>
__global__ __launch_bounds__(RS::L ? kRowThreads : 1024) void residual_fwd(FwdP p) {
    constexpr int L = RS::L, NC = RS::NC, U = units_per_block<L>();
    constexpr Ends RAGGED = RS::RAGGED;
    __shared__ SumMemory<L, NC, false> lds;
    const RowLane<RS> lane(1, p.W);
    const Groups groups{1, 0};
    const int n = p.W;
    struct Row {
        Piece<T> b[NC];
        Piece<R> r[NC];
    };
    int64_t row = (int64_t)blockIdx.x * U + lane.ul.unit;
    const int64_t stride = (int64_t)p.slices * U;
    RowPtr<T> b(p.b, p.ld_x, row, 0), h(p.h, p.ld_out, row, 0);
    RowPtr<R> r(p.r, p.ld_res, row, 0), r_out(p.r_out, p.ld_res, row, 0);
    CkptRow r8(p.r8, p.scale_off, p.W32, row, 0), b8(p.b8, p.scale_off, p.W32, row, 0), h8(p.h8, p.scale_off, p.W32, row, 0);
    auto load = [&](Row& o) {
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            if (p.b) load8<RAGGED>(o.b[k], b.p, lane.at(k), n);
            if (p.r) load8<RAGGED>(o.r[k], r.p, lane.at(k), n);
        }
    };
    // what is not given, and lanes past the width, keep the zeros of the start
    Row next = {};
    Piece<float> w[NC] = {}, e[NC];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        fetch8<RAGGED>(w[k], p.w, lane.at(k), n);
        e[k] = branch_factor<RAGGED>(p.w_post, p.scale, p.alpha, lane.at(k), n);
    }
    lds.init();
    if (row < p.M) load(next);
    int turn = 0;
    walk_rows(next, row - lane.ul.unit, p.M, stride, [&](Row& o, Row& next) {
        b.skip(stride);
        r.skip(stride);
        if (row + stride < p.M) load(next);
        const bool valid = row < p.M;
        float x[NC][8], ss[NC], post[NC], rstd[NC];
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            settle8<RAGGED>(o.b[k], lane.at(k), n);
            settle8<RAGGED>(o.r[k], lane.at(k), n);
            post[k] = 1.0f;
        }
        if (p.w_post) {
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                ss[k] = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) ss[k] += o.b[k][j] * o.b[k][j];
            }
            unit_rstd(ss, [&](int k, int j) { return o.b[k][j]; }, post, lds, turn, lane.group, groups, p.inv_n, p.eps);
            if (valid && p.rstd_post && lane.ul.lane == 0) p.rstd_post[row] = post[0];
        }
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            ss[k] = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[k][j] = o.r[k][j] + (o.b[k][j] * post[k]) * e[k][j];
                ss[k] += x[k][j] * x[k][j];
            }
        }
        unit_rstd(ss, [&](int k, int j) { return x[k][j]; }, rstd, lds, turn, lane.group, groups, p.inv_n, p.eps);
        if (valid) {
            if (p.rstd && lane.ul.lane == 0) p.rstd[row] = rstd[0];
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                const int at = lane.at(k);
                float y[8], v[8];
                if (p.r_out) store8<RAGGED>(r_out.p, at, n, x[k]);
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = x[k][j] * rstd[0] * w[k][j];
                store8<RAGGED>(h.p, at, n, y);
                if (at >= p.W32) continue;
                if (p.r8) {
                    as_stored<R>(x[k], v);
                    r8.store(at, v);
                }
                if (p.b8) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = o.b[k][j];
                    b8.store(at, v);
                }
                if (p.h8) {
                    as_stored<T>(y, v);
                    h8.store(at, v);
                }
            }
        }
        row += stride;
        r_out.skip(stride);
        h.skip(stride);
        r8.skip(stride);
        b8.skip(stride);
        h8.skip(stride);
    });
}

}  // namespace

int launch_norm_residual_fwd(const ResidualArgs& a, hipStream_t stream) {
    const NormShape& s = a.s;
    if (!s.M) return SSM_OK;
    return for_row_shape<kResidual>(s.M, s.W, 1, [&](auto rs, int threads, int) {
        using RS = decltype(rs);
        const int slices = row_slices<RS>(s.M, 1, threads);
        FwdP p = {a.b, a.r, a.w_post, a.scale, a.w, a.r_out, a.h, a.rstd, a.rstd_post, a.r8, a.b8, a.h8, s.ld_x,
                  s.ld_res, s.ld_out, s.M, s.scale_off, s.W, s.W32, slices, s.eps, 1.0f / (float)s.W, s.alpha};
        for_types(s, [&](auto t, auto r) {
            residual_fwd<decltype(t), decltype(r), RS><<<slices, threads, 0, stream>>>(p);
        });
        return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
    });
}

}  // namespace ssm
