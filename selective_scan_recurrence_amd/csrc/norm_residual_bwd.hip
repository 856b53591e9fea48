// Backward of the residual norm (norm_residual.hip has the formulas), and the
// sums over rows of both norms: each workgroup of a backward adds the rows of
// its slice in registers and stores one partial row; column_sums adds the
// partial rows in a fixed order.  Bound by HBM.
#include "norm_residual.h"

namespace ssm {
namespace {

struct BwdP {
    const void *dh, *dr_out, *r_out, *b;
    uint8_t *r8, *b8;
    const float *w_post, *scale, *w, *rstd, *rstd_post;
    void *d_r, *d_b;
    float *part_w, *part_s;  // [slices][W] each, or null
    int64_t ld_x, ld_res, ld_out, M, scale_off;
    int W, W32, slices;
    float inv_n, alpha;
};

// BRANCH: b takes part (a norm after the block, or the scale's gradient)
template <typename T, typename R, typename RS, bool BRANCH>
__global__ __launch_bounds__(RS::L ? kRowThreads : 1024) void residual_bwd(BwdP p) {
    constexpr int L = RS::L, NC = RS::NC, NB = BRANCH ? NC : 1, U = units_per_block<L>();
    constexpr Ends RAGGED = RS::RAGGED;
    __shared__ SumMemory<L, NC, false> lds;
    __shared__ float sm[L ? kRowThreads * 8 : 1];
    const RowLane<RS> lane(1, p.W);
    const Groups groups{1, 0};
    const int n = p.W;
    struct Row {
        Piece<T> dh[NC];
        Piece<R> dr[NC];
        PieceOr8<R> r[NC];
        PieceOr8<T> b[NB];
        float rstd, post;
    };
    int64_t row = (int64_t)blockIdx.x * U + lane.ul.unit;
    const int64_t stride = (int64_t)p.slices * U;
    RowPtr<T> dh(p.dh, p.ld_out, row, 0), b(p.b, p.ld_x, row, 0), d_b(p.d_b, p.ld_x, row, 0);
    RowPtr<R> r_out(p.r_out, p.ld_res, row, 0), dr_out(p.dr_out, p.ld_res, row, 0), d_r(p.d_r, p.ld_res, row, 0);
    CkptRow r8(p.r8, p.scale_off, p.W32, row, 0), b8(p.b8, p.scale_off, p.W32, row, 0);
    auto load = [&](Row& o, int64_t of) {
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int at = lane.at(k);
            load8<RAGGED>(o.dh[k], dh.p, at, n);
            if (!p.r8) load8<RAGGED>(o.r[k].t, r_out.p, at, n);
            else if (at < n) o.r[k].c = r8.load(at);
            if (p.dr_out) load8<RAGGED>(o.dr[k], dr_out.p, at, n);
            if constexpr (BRANCH) {
                if (!p.b8) load8<RAGGED>(o.b[k].t, b.p, at, n);
                else if (at < n) o.b[k].c = b8.load(at);
            }
        }
        o.rstd = p.rstd[of];
        o.post = BRANCH && p.w_post ? p.rstd_post[of] : 1.0f;
    };
    Row next;
    __builtin_memset(&next, 0, sizeof next);
    Piece<float> w[NC] = {}, e[NC];
    float dw[NC][8], ds[NB][8];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        fetch8<RAGGED>(w[k], p.w, lane.at(k), n);
        e[k] = branch_factor<RAGGED>(p.w_post, p.scale, p.alpha, lane.at(k), n);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dw[k][j] = 0.0f;
            if (BRANCH) ds[k][j] = 0.0f;
        }
    }
    lds.init();
    if (row < p.M) load(next, row);
    int turn = 0;
    walk_rows(next, row - lane.ul.unit, p.M, stride, [&](Row& o, Row& next) {
        dh.skip(stride);
        r_out.skip(stride);
        dr_out.skip(stride);
        b.skip(stride);
        r8.skip(stride);
        b8.skip(stride);
        if (row + stride < p.M) load(next, row + stride);
        const bool valid = row < p.M;  // else o is an earlier row: it is not counted again
        float x[NC][8], dot[NC], c1[NC];
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            settle8<RAGGED>(o.dh[k], lane.at(k), n);
            settle8<RAGGED>(o.dr[k], lane.at(k), n);
            o.r[k].template values<RAGGED>(p.r8, x[k], lane.at(k), n);
            dot[k] = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[k][j] *= o.rstd;
                const float dx = o.dh[k][j] * x[k][j];
                if (valid) dw[k][j] += dx;
                dot[k] += dx * w[k][j];
            }
        }
        unit_sum(dot, c1, lds, turn++, lane.group, groups);
        c1[0] *= p.inv_n;
        // x becomes dx, then dm
        float v[NB][8];
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            dot[k] = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[k][j] = o.rstd * (o.dh[k][j] * w[k][j] - x[k][j] * c1[0]) + o.dr[k][j];
            if (valid && p.d_r) store8<RAGGED>(d_r.p, lane.at(k), n, x[k]);
            if constexpr (BRANCH) {
                o.b[k].template values<RAGGED>(p.b8, v[k], lane.at(k), n);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[k][j] *= o.post;
                    if (valid) ds[k][j] += x[k][j] * v[k][j];
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[k][j] *= e[k][j];
                if (BRANCH) dot[k] += x[k][j] * v[k][j];
            }
        }
        if (BRANCH && p.w_post) {
            float c2[NC];
            unit_sum(dot, c2, lds, turn++, lane.group, groups);
            c2[0] *= p.inv_n;
#pragma unroll
            for (int k = 0; k < NC; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) x[k][j] = o.post * (x[k][j] - v[k][j] * c2[0]);
        }
        if (valid && p.d_b)
#pragma unroll
            for (int k = 0; k < NC; ++k) store8<RAGGED>(d_b.p, lane.at(k), n, x[k]);
        row += stride;
        d_r.skip(stride);
        d_b.skip(stride);
    });
    const int64_t part = (int64_t)blockIdx.x * p.W;
    if (p.part_w) store_column_sums<L, NC, RAGGED>(p.part_w + part, n, dw, sm);
    if constexpr (BRANCH)
        if (p.part_s) store_column_sums<L, NC, RAGGED>(p.part_s + part, n, ds, sm);
}

// Sums S partial rows: 32 columns (a cache line) a workgroup, 32 lanes down the
// rows.  Array
// 0 gives d_w; array 1 the S of the note above, hence d_w_post and d_scale.
struct SumP {
    ColumnSums o;
    const float* part;
    int S, W;
};
constexpr int kSumCols = 32, kSumRows = 32;
__global__ __launch_bounds__(kSumCols* kSumRows) void column_sums(SumP p) {
    __shared__ float sm[kSumRows][kSumCols];
    const int c = threadIdx.x % kSumCols, l = threadIdx.x / kSumCols;
    const int col = blockIdx.x * kSumCols + c;
    const float* part = p.part + (int64_t)blockIdx.y * p.S * p.W;
    float v = 0.0f;
    if (col < p.W)
#pragma unroll 4
        for (int s = l; s < p.S; s += kSumRows) v += part[(int64_t)s * p.W + col];
    sm[l][c] = v;
    __syncthreads();
    for (int h = kSumRows / 2; h > 0; h /= 2) {
        if (l < h) sm[l][c] += sm[l + h][c];
        __syncthreads();
    }
    if (l != 0 || col >= p.W) return;
    v = sm[0][c];
    if (blockIdx.y == 0) {
        if (p.o.d_w) p.o.d_w[col] = v;
    } else {
        v *= p.o.alpha;
        if (p.o.d_w_post) p.o.d_w_post[col] = p.o.scale ? v * p.o.scale[col] : v;
        if (p.o.d_scale) p.o.d_scale[col] = p.o.w_post ? v * p.o.w_post[col] : v;
    }
}

}  // namespace

// A unit of a workgroup takes at least 2 rows, and the workgroups are those that
// 256 compute units hold at a time with 4 waves on each SIMD (2 for a wave with
// more than one piece), where a workgroup of more than 4 waves counts as if it
// filled its last four.  That is what 128 registers a lane (256) leave room for:
// the residual norm with the branch takes up to 171, and with three pieces up to
// 374 in all but the bf16 form without the branch, so that theirs run in more
// rounds than one.  Beyond 768 of them
// there are only as many as leave 16 rows for each, so that the partial sums stay few
// beside the rows.  (Gated backward of 65536 rows in bf16, times of a copy's:
// width 2560, 5 waves, 1.66, 1.08, 1.38 with 1, 2, 3 workgroups on a unit; width
// 1280, 3 waves, 1.35, 1.13, 1.01, 1.35 with 3 to 6; width 2048, 4 waves, 0.93,
// 0.88, 1.18 with 3 to 5.  1111 x 771 f32, gate after: 8.5, 9.4, 13.5, 21.4 us
// with 1, 2, 4, 8 rows, where the sum of the partial rows grows from 2 to 5 us
// with 1.)
int norm_bwd_slices(const NormShape& s, bool gated) {
    int rows = 1;
    int64_t most = 1;
    auto count = [&](auto rs, int threads, int units) {
        using RS = decltype(rs);
        rows = 2 * units_per_block<RS::L>();
        const int waves = threads / 64, simds = (waves + 3) / 4;
        const int each = RS::L && RS::NC > 1 ? 2 : waves <= 4 ? 16 / waves : 4 / simds;
        most = 256 * each / units;
        return 0;
    };
    if (gated) for_row_shape<kGatedBwd>(s.M, s.W, s.G, count);
    else for_row_shape<kResidual>(s.M, s.W, 1, count);
    const int64_t cap = s.M / 16 > 768 ? s.M / 16 : 768;
    most = most < 1 ? 1 : most > cap ? cap : most;
    const int64_t want = (s.M + rows - 1) / rows;
    return (int)(want < 1 ? 1 : want < most ? want : most);
}

int launch_column_sums(const float* part, int S, int W, const ColumnSums& out, hipStream_t stream) {
    SumP p = {out, part, S, W};
    column_sums<<<dim3((W + kSumCols - 1) / kSumCols, out.d_w_post || out.d_scale ? 2 : 1), kSumCols * kSumRows, 0,
                  stream>>>(p);
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int launch_norm_residual_bwd(const ResidualBwdArgs& a, hipStream_t stream) {
    const NormShape& s = a.s;
    const int slices = norm_bwd_slices(s, false);
    const bool branch = a.w_post || a.d_scale, sums = a.d_w_post || a.d_scale;
    const bool direct = slices == 1 && !sums;  // d_w is the one partial row
    float* part_w = direct ? a.d_w : a.d_w || sums ? a.part : nullptr;
    BwdP p = {a.dh, a.dr_out, a.r_out, a.b, const_cast<uint8_t*>(a.r8), const_cast<uint8_t*>(a.b8), a.w_post,
              a.scale, a.w, a.rstd, a.rstd_post, a.d_r, a.d_b, part_w,
              sums ? a.part + (int64_t)slices * s.W : nullptr, s.ld_x, s.ld_res, s.ld_out, s.M, s.scale_off, s.W,
              s.W32, slices, 1.0f / (float)s.W, s.alpha};
    const int rc = for_row_shape<kResidual>(s.M, s.W, 1, [&](auto rs, int threads, int) {
        using RS = decltype(rs);
        for_types(s, [&](auto t, auto r) {
            using T = decltype(t);
            using R = decltype(r);
            if (branch) residual_bwd<T, R, RS, true><<<slices, threads, 0, stream>>>(p);
            else residual_bwd<T, R, RS, false><<<slices, threads, 0, stream>>>(p);
        });
        return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
    });
    if (rc != SSM_OK || direct || !part_w) return rc;
    return launch_column_sums(a.part, slices, s.W, ColumnSums{a.d_w, a.d_w_post, a.d_scale, a.scale, a.w_post, s.alpha},
                              stream);
}

}  // namespace ssm
