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
// held in registers between its sums and the outputs (norm_rows.h).  The
// column sums over rows also keep this file's last kernel: each workgroup of a
// backward adds the rows of its slice in registers and stores one partial row;
// column_sums adds the partial rows in a fixed order.
#include "block_internal.h"
#include "norm_rows.h"

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

// e of this lane's pieces
template <bool RAGGED>
__device__ __forceinline__ Piece<float> branch_factor(const float* w_post, const float* scale, float alpha, int at, int n) {
    Piece<float> e = {}, t = {};
#pragma unroll
    for (int j = 0; j < 8; ++j) e.d[j] = alpha;
    if (scale) {
        load8<RAGGED>(t, scale, at, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) e.d[j] *= t.d[j];
    }
    if (w_post) {
        load8<RAGGED>(t, w_post, at, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) e.d[j] *= t.d[j];
    }
    return e;
}

// Workgroup i takes every slices-th row (or set of rows) from i on, and loads
// the next one while it works on the present one.
template <typename T, typename R, int L, int NC, bool RAGGED>
__global__ __launch_bounds__(L ? kRowThreads : 1024) void residual_fwd(FwdP p) {
    __shared__ float lds[32];
    constexpr int U = units_per_block<L>();
    const UnitLane ul = unit_lane<L>();
    const int n = p.W;
    const T* b = static_cast<const T*>(p.b);
    const R* r_in = static_cast<const R*>(p.r);
    R* r_out = static_cast<R*>(p.r_out);
    T* h = static_cast<T*>(p.h);
    const Ckpt r8(p.r8, p.scale_off, p.W32, 0), b8(p.b8, p.scale_off, p.W32, 0), h8(p.h8, p.scale_off, p.W32, 0);
    struct Row {
        Piece<T> b[NC];
        Piece<R> r[NC];
    };
    auto load = [&](Row& o, int64_t row) {
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            if (p.b) load8<RAGGED>(o.b[k], b + row * p.ld_x, ul.at(k), n);
            if (p.r) load8<RAGGED>(o.r[k], r_in + row * p.ld_res, ul.at(k), n);
        }
    };
    // what is not given, and lanes past the width, keep the zeros of the start
    Row next = {};
    Piece<float> w[NC] = {}, e[NC];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        load8<RAGGED>(w[k], p.w, ul.at(k), n);
        e[k] = branch_factor<RAGGED>(p.w_post, p.scale, p.alpha, ul.at(k), n);
    }
    unit_sum_init<L>(lds);
    int64_t row = (int64_t)blockIdx.x * U + ul.unit;
    const int64_t step = (int64_t)p.slices * U;
    if (row < p.M) load(next, row);
    int turn = 0;
    for (int64_t first = row - ul.unit; first < p.M; first += step, row += step) {
        const Row o = next;
        if (row + step < p.M) load(next, row + step);
        const bool valid = row < p.M;
        float post = 1.0f;
        if (p.w_post) {
            float ss = 0.0f;
#pragma unroll
            for (int k = 0; k < NC; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) ss += o.b[k][j] * o.b[k][j];
            post = rsqrt1(unit_sum<L>(ss, lds, turn++) * p.inv_n + p.eps);
            if (valid && p.rstd_post && ul.lane == 0) p.rstd_post[row] = post;
        }
        float x[NC][8], ss = 0.0f;
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[k][j] = o.r[k][j] + (o.b[k][j] * post) * e[k][j];
                ss += x[k][j] * x[k][j];
            }
        const float rstd = rsqrt1(unit_sum<L>(ss, lds, turn++) * p.inv_n + p.eps);
        if (!valid) continue;
        if (p.rstd && ul.lane == 0) p.rstd[row] = rstd;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            float y[8], v[8];
            if (r_out) store8<RAGGED>(r_out + row * p.ld_res, ul.at(k), n, x[k]);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = x[k][j] * rstd * w[k][j];
            store8<RAGGED>(h + row * p.ld_out, ul.at(k), n, y);
            if (ul.at(k) >= p.W32) continue;
            if (p.r8) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = as_stored(x[k][j], R());
                r8.store(row, ul.at(k), v);
            }
            if (p.b8) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = o.b[k][j];
                b8.store(row, ul.at(k), v);
            }
            if (p.h8) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = as_stored(y[j], T());
                h8.store(row, ul.at(k), v);
            }
        }
    }
}

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
template <typename T, typename R, int L, int NC, bool RAGGED, bool BRANCH>
__global__ __launch_bounds__(L ? kRowThreads : 1024) void residual_bwd(BwdP p) {
    __shared__ float lds[L ? kRowThreads * 8 : 32];
    constexpr int U = units_per_block<L>(), NB = BRANCH ? NC : 1;
    const UnitLane ul = unit_lane<L>();
    const int n = p.W;
    const T* dh = static_cast<const T*>(p.dh);
    const T* b = static_cast<const T*>(p.b);
    const R* r_out = static_cast<const R*>(p.r_out);
    const R* dr_out = static_cast<const R*>(p.dr_out);
    R* d_r = static_cast<R*>(p.d_r);
    T* d_b = static_cast<T*>(p.d_b);
    const Ckpt r8(p.r8, p.scale_off, p.W32, 0), b8(p.b8, p.scale_off, p.W32, 0);
    struct Row {
        Piece<T> dh[NC];
        Piece<R> dr[NC];
        PieceOr8<R> r[NC];
        PieceOr8<T> b[NB];
        float rstd, post;
    };
    auto load = [&](Row& o, int64_t row) {
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            load8<RAGGED>(o.dh[k], dh + row * p.ld_out, ul.at(k), n);
            if (!p.r8) load8<RAGGED>(o.r[k].t, r_out + row * p.ld_res, ul.at(k), n);
            else if (ul.at(k) < n) o.r[k].c = r8.load(row, ul.at(k));
            if (p.dr_out) load8<RAGGED>(o.dr[k], dr_out + row * p.ld_res, ul.at(k), n);
            if constexpr (BRANCH) {
                if (!p.b8) load8<RAGGED>(o.b[k].t, b + row * p.ld_x, ul.at(k), n);
                else if (ul.at(k) < n) o.b[k].c = b8.load(row, ul.at(k));
            }
        }
        o.rstd = p.rstd[row];
        o.post = BRANCH && p.w_post ? p.rstd_post[row] : 1.0f;
    };
    Row next;
    __builtin_memset(&next, 0, sizeof next);
    Piece<float> w[NC] = {}, e[NC];
    float dw[NC][8], ds[NB][8];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        load8<RAGGED>(w[k], p.w, ul.at(k), n);
        e[k] = branch_factor<RAGGED>(p.w_post, p.scale, p.alpha, ul.at(k), n);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dw[k][j] = 0.0f;
            if (BRANCH) ds[k][j] = 0.0f;
        }
    }
    unit_sum_init<L>(lds);
    int64_t row = (int64_t)blockIdx.x * U + ul.unit;
    const int64_t step = (int64_t)p.slices * U;
    if (row < p.M) load(next, row);
    int turn = 0;
    for (int64_t first = row - ul.unit; first < p.M; first += step, row += step) {
        const Row o = next;
        if (row + step < p.M) load(next, row + step);
        const bool valid = row < p.M;  // else o is the row before: it is not counted again
        float x[NC][8], dot = 0.0f;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            if (p.r8) o.r[k].c.values(x[k]);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) x[k][j] = o.r[k].t[j];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[k][j] *= o.rstd;
                const float dx = o.dh[k][j] * x[k][j];
                if (valid) dw[k][j] += dx;
                dot += dx * w[k][j];
            }
        }
        const float c1 = unit_sum<L>(dot, lds, turn++) * p.inv_n;
        // x becomes dx, then dm
        float v[NB][8], dot2 = 0.0f;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[k][j] = o.rstd * (o.dh[k][j] * w[k][j] - x[k][j] * c1) + o.dr[k][j];
            if (valid && d_r) store8<RAGGED>(d_r + row * p.ld_res, ul.at(k), n, x[k]);
            if constexpr (BRANCH) {
                if (p.b8) o.b[k].c.values(v[k]);
                else
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[k][j] = o.b[k].t[j];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[k][j] *= o.post;
                    if (valid) ds[k][j] += x[k][j] * v[k][j];
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[k][j] *= e[k][j];
                if (BRANCH) dot2 += x[k][j] * v[k][j];
            }
        }
        if (BRANCH && p.w_post) {
            const float c2 = unit_sum<L>(dot2, lds, turn++) * p.inv_n;
#pragma unroll
            for (int k = 0; k < NC; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) x[k][j] = o.post * (x[k][j] - v[k][j] * c2);
        }
        if (valid && d_b)
#pragma unroll
            for (int k = 0; k < NC; ++k) store8<RAGGED>(d_b + row * p.ld_x, ul.at(k), n, x[k]);
    }
    const int64_t part = (int64_t)blockIdx.x * p.W;
    if (p.part_w) store_column_sums<L, NC, RAGGED>(p.part_w + part, n, dw, lds);
    if constexpr (BRANCH)
        if (p.part_s) store_column_sums<L, NC, RAGGED>(p.part_s + part, n, ds, lds);
}

// Sums S partial rows: 16 columns a workgroup, 64 lanes down the rows.  Array
// 0 gives d_w; array 1 the S of the note above, hence d_w_post and d_scale.
struct SumP {
    ColumnSums o;
    const float* part;
    int S, W;
};
constexpr int kSumCols = 16, kSumRows = 64;
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

template <typename F>
void for_types(const NormShape& s, F&& f) {
    if (s.io == SSM_F32) f(float(), float());
    else if (s.res == SSM_F32) f(bf16_t(), float());
    else f(bf16_t(), bf16_t());
}

}  // namespace

// A unit of a workgroup takes at least 2 rows, and there are at most 768
// workgroups over all groups, so that the partial sums stay few beside the
// rows.  (1111 x 771 f32, gate after: 8.5, 9.4, 13.5, 21.4 us with 1, 2, 4, 8
// rows, where the sum of the partial rows grows from 2 to 5 us with 1.  At
// 16384 x 2560, 512 and 768 workgroups are alike, 1024 are 5% slower.)
int norm_bwd_slices(const NormShape& s) {
    int upb = 1;
    for_row_shape(s.Wg, [&](auto rs) { upb = units_per_block<decltype(rs)::L>(); return 0; });
    const int64_t want = (s.M + 2 * (int64_t)upb - 1) / (2 * (int64_t)upb);
    const int64_t most = 768 / s.G > 0 ? 768 / s.G : 1;
    return (int)(want < 1 ? 1 : want < most ? want : most);
}

int launch_column_sums(const float* part, int S, int W, const ColumnSums& out, hipStream_t stream) {
    SumP p = {out, part, S, W};
    column_sums<<<dim3((W + kSumCols - 1) / kSumCols, out.d_w_post || out.d_scale ? 2 : 1), kSumCols * kSumRows, 0,
                  stream>>>(p);
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int launch_norm_residual_fwd(const ResidualArgs& a, hipStream_t stream) {
    const NormShape& s = a.s;
    if (!s.M) return SSM_OK;
    return for_row_shape(s.W, [&](auto rs) {
        using RS = decltype(rs);
        const int threads = row_threads<RS>(s.W), slices = row_slices<RS>(s.M, 1, threads);
        FwdP p = {a.b, a.r, a.w_post, a.scale, a.w, a.r_out, a.h, a.rstd, a.rstd_post, a.r8, a.b8, a.h8, s.ld_x,
                  s.ld_res, s.ld_out, s.M, s.scale_off, s.W, s.W32, slices, s.eps, 1.0f / (float)s.W, s.alpha};
        for_types(s, [&](auto t, auto r) {
            residual_fwd<decltype(t), decltype(r), RS::L, RS::NC, RS::RAGGED><<<slices, threads, 0, stream>>>(p);
        });
        return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
    });
}

int launch_norm_residual_bwd(const ResidualBwdArgs& a, hipStream_t stream) {
    const NormShape& s = a.s;
    const int slices = norm_bwd_slices(s);
    const bool branch = a.w_post || a.d_scale, sums = a.d_w_post || a.d_scale;
    const bool direct = slices == 1 && !sums;  // d_w is the one partial row
    float* part_w = direct ? a.d_w : a.d_w || sums ? a.part : nullptr;
    BwdP p = {a.dh, a.dr_out, a.r_out, a.b, const_cast<uint8_t*>(a.r8), const_cast<uint8_t*>(a.b8), a.w_post,
              a.scale, a.w, a.rstd, a.rstd_post, a.d_r, a.d_b, part_w,
              sums ? a.part + (int64_t)slices * s.W : nullptr, s.ld_x, s.ld_res, s.ld_out, s.M, s.scale_off, s.W,
              s.W32, slices, 1.0f / (float)s.W, s.alpha};
    const int rc = for_row_shape(s.W, [&](auto rs) {
        using RS = decltype(rs);
        const int threads = row_threads<RS>(s.W);
        for_types(s, [&](auto t, auto r) {
            using T = decltype(t);
            using R = decltype(r);
            if (branch) residual_bwd<T, R, RS::L, RS::NC, RS::RAGGED, true><<<slices, threads, 0, stream>>>(p);
            else residual_bwd<T, R, RS::L, RS::NC, RS::RAGGED, false><<<slices, threads, 0, stream>>>(p);
        });
        return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
    });
    if (rc != SSM_OK || direct || !part_w) return rc;
    return launch_column_sums(a.part, slices, s.W, ColumnSums{a.d_w, a.d_w_post, a.d_scale, a.scale, a.w_post, s.alpha},
                              stream);
}

}  // namespace ssm
