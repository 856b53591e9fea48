// The norm between two blocks, forward and backward.  Per row:
//   t  = b,  or  b rstd_post w_post  (norm after the block)
//   r' = r + alpha scale t           (residual add and scale)
//   h  = r' rstd w                   (norm before the next block)
// with rstd = 1 / sqrt(mean r'^2 + eps), rstd_post the same of b; and, with
// c() the mean over the row:
//   x  = r' rstd, dn = dh w, dx = rstd (dn - x c(dn x)) + d_r_out,  d_r = dx
//   dt = alpha scale dx;  dw = sum_rows dh x;  dscale = sum_rows alpha dx t
//   with the norm after the block: v = b rstd_post, dm = dt w_post,
//     db = rstd_post (dm - v c(dm v)), dw_post = sum_rows dt v;  else db = dt
// All of it in f32; what is stored in fewer bits is rounded once.
//
// Bound by HBM: each input is read once and each output written once, the row
// held in registers between its sums and the outputs (norm_rows.h).  The
// column sums over rows also keep this file's second kernel: each workgroup
// of the backward adds the rows of its slice in registers and stores one
// partial row; column_sums adds the partial rows in a fixed order.
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
    int W, W32;
    float eps, inv_n, alpha;
};

template <typename T, typename R, int L, int NC>
__global__ __launch_bounds__(L ? kRowThreads : 1024) void residual_fwd(FwdP p) {
    __shared__ float lds[32];
    const UnitLane ul = unit_lane<L>();
    const int64_t id = block_id() * units_per_block<L>() + ul.unit;
    const bool valid = id < p.M;
    const int64_t row = valid ? id : 0;
    const int W = valid ? p.W : 0;
    const T* b = p.b ? static_cast<const T*>(p.b) + row * p.ld_x : nullptr;
    const R* r = p.r ? static_cast<const R*>(p.r) + row * p.ld_res : nullptr;
    float bv[NC][8], x[NC][8];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = ul.lane + k * ul.lanes, n = W - 8 * c;
#pragma unroll
        for (int j = 0; j < 8; ++j) bv[k][j] = x[k][j] = 0.0f;
        if (n > 0) {
            if (b) {
                const Piece<T> t = load8(b + 8 * c, n);
#pragma unroll
                for (int j = 0; j < 8; ++j) bv[k][j] = t[j];
            }
            if (r) {
                const Piece<R> t = load8(r + 8 * c, n);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[k][j] = t[j];
            }
        }
    }
    float post = 1.0f;
    if (p.w_post) {
        float ss = 0.0f;
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss += bv[k][j] * bv[k][j];
        post = 1.0f / sqrtf(unit_sum<L>(ss, lds, 0) * p.inv_n + p.eps);
        if (valid && p.rstd_post && ul.lane == 0) p.rstd_post[row] = post;
    }
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = ul.lane + k * ul.lanes, n = W - 8 * c;
        float t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = p.w_post ? bv[k][j] * post : bv[k][j];
        if (n > 0 && p.w_post) {
            const Piece<float> w = load8(p.w_post + 8 * c, n);
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] *= w[j];
        }
        if (n > 0 && p.scale) {
            const Piece<float> w = load8(p.scale + 8 * c, n);
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] *= w[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[k][j] += p.alpha * t[j];
            ss += x[k][j] * x[k][j];
        }
    }
    const float rstd = 1.0f / sqrtf(unit_sum<L>(ss, lds, 1) * p.inv_n + p.eps);
    if (valid && p.rstd && ul.lane == 0) p.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = ul.lane + k * ul.lanes, n = W - 8 * c;
        float h[8] = {};
        if (n > 0) {
            if (p.r_out) store8(static_cast<R*>(p.r_out) + row * p.ld_res + 8 * c, n, x[k]);
            const Piece<float> w = load8(p.w + 8 * c, n);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] = x[k][j] * rstd * w[j];
            store8(static_cast<T*>(p.h) + row * p.ld_out + 8 * c, n, h);
        }
        if (8 * c < (valid ? p.W32 : 0)) {
            float v[8];
            if (p.r8) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = as_stored(x[k][j], R());
                ckpt_store(ckpt_row(p.r8, p.scale_off, p.W32, row, 0), c, v);
            }
            if (p.b8) ckpt_store(ckpt_row(p.b8, p.scale_off, p.W32, row, 0), c, bv[k]);
            if (p.h8) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = as_stored(h[j], T());
                ckpt_store(ckpt_row(p.h8, p.scale_off, p.W32, row, 0), c, v);
            }
        }
    }
}

struct BwdP {
    const void *dh, *dr_out, *r_out, *b;
    uint8_t *r8, *b8;
    const float *w_post, *scale, *w, *rstd, *rstd_post;
    void *d_r, *d_b;
    float *part_w, *part_post, *part_scale;  // [slices][W] each, or null
    int64_t ld_x, ld_res, ld_out, M, scale_off;
    int W, W32, slices;
    float inv_n, alpha;
};

// BR: the branch b takes part (norm after the block, or the scale's gradient)
template <typename T, typename R, int L, int NC, bool BR>
__global__ __launch_bounds__(L ? kRowThreads : 1024) void residual_bwd(BwdP p) {
    __shared__ float lds[L ? kRowThreads * 8 : 32];
    const UnitLane ul = unit_lane<L>();
    float dw[NC][8], dwp[BR ? NC : 1][8], ds[BR ? NC : 1][8];
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dw[k][j] = 0.0f;
            if (BR) dwp[k][j] = ds[k][j] = 0.0f;
        }
    int turn = 0;
    const int64_t step = (int64_t)p.slices * units_per_block<L>();
    for (int64_t r0 = (int64_t)blockIdx.x * units_per_block<L>(); r0 < p.M; r0 += step) {
        const int64_t row = r0 + ul.unit;
        const bool valid = row < p.M;
        const int W = valid ? p.W : 0;
        const int64_t rr = valid ? row : 0;
        const float rstd = valid ? p.rstd[rr] : 0.0f;
        float x[NC][8], dn[NC][8], dx[NC][8], v[BR ? NC : 1][8], dot = 0.0f;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int c = ul.lane + k * ul.lanes, n = W - 8 * c;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[k][j] = dn[k][j] = dx[k][j] = 0.0f;
                if (BR) v[k][j] = 0.0f;
            }
            if (n <= 0) continue;
            const Piece<T> d = load8(static_cast<const T*>(p.dh) + rr * p.ld_out + 8 * c, n);
            if (p.r8) {
                ckpt_load(ckpt_row(p.r8, p.scale_off, p.W32, rr, 0), c, x[k]);
            } else {
                const Piece<R> t = load8(static_cast<const R*>(p.r_out) + rr * p.ld_res + 8 * c, n);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[k][j] = t[j];
            }
            if (p.dr_out) {
                const Piece<R> t = load8(static_cast<const R*>(p.dr_out) + rr * p.ld_res + 8 * c, n);
#pragma unroll
                for (int j = 0; j < 8; ++j) dx[k][j] = t[j];
            }
            if constexpr (BR) {
                if (p.b8) {
                    ckpt_load(ckpt_row(p.b8, p.scale_off, p.W32, rr, 0), c, v[k]);
                } else {
                    const Piece<T> t = load8(static_cast<const T*>(p.b) + rr * p.ld_x + 8 * c, n);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[k][j] = t[j];
                }
            }
            const Piece<float> w = load8(p.w + 8 * c, n);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[k][j] *= rstd;
                dw[k][j] += d[j] * x[k][j];
                dn[k][j] = d[j] * w[j];
                dot += dn[k][j] * x[k][j];
            }
        }
        const float c1 = unit_sum<L>(dot, lds, turn++) * p.inv_n;
        const float post = BR && p.w_post && valid ? p.rstd_post[rr] : 1.0f;
        float dot2 = 0.0f;
        // dn becomes dt, then (norm after the block) dm = dt w_post
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int c = ul.lane + k * ul.lanes, n = W - 8 * c;
            if (n <= 0) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) dx[k][j] += rstd * (dn[k][j] - x[k][j] * c1);
            if (p.d_r) store8(static_cast<R*>(p.d_r) + rr * p.ld_res + 8 * c, n, dx[k]);
            Piece<float> sc, wp;
            if (p.scale) sc = load8(p.scale + 8 * c, n);
            if (BR && p.w_post) wp = load8(p.w_post + 8 * c, n);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float adx = p.alpha * dx[k][j];
                dn[k][j] = p.scale ? adx * sc[j] : adx;
                if constexpr (BR) {
                    v[k][j] *= post;
                    ds[k][j] += adx * (p.w_post ? v[k][j] * wp[j] : v[k][j]);
                    if (p.w_post) {
                        dwp[k][j] += dn[k][j] * v[k][j];
                        dn[k][j] *= wp[j];
                        dot2 += dn[k][j] * v[k][j];
                    }
                }
            }
        }
        if (BR && p.w_post) {
            const float c2 = unit_sum<L>(dot2, lds, turn++) * p.inv_n;
#pragma unroll
            for (int k = 0; k < NC; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) dn[k][j] = post * (dn[k][j] - v[k][j] * c2);
        }
        if (p.d_b)
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                const int c = ul.lane + k * ul.lanes, n = W - 8 * c;
                if (n > 0) store8(static_cast<T*>(p.d_b) + rr * p.ld_x + 8 * c, n, dn[k]);
            }
    }
    const int64_t at = (int64_t)blockIdx.x * p.W;
    if (p.part_w) store_column_sums<L, NC>(p.part_w + at, p.W, dw, lds);
    if constexpr (BR) {
        if (p.part_post) store_column_sums<L, NC>(p.part_post + at, p.W, dwp, lds);
        if (p.part_scale) store_column_sums<L, NC>(p.part_scale + at, p.W, ds, lds);
    }
}

// out[c] = sum_s part[s][c]: 16 columns a workgroup, 64 lanes down the rows.
struct SumP {
    const float* part;
    float* out[3];
    int S, W;
};
constexpr int kSumCols = 16, kSumRows = 64;
__global__ __launch_bounds__(kSumCols* kSumRows) void column_sums(SumP p) {
    __shared__ float sm[kSumRows][kSumCols];
    const int c = threadIdx.x % kSumCols, l = threadIdx.x / kSumCols;
    const int col = blockIdx.x * kSumCols + c;
    float* out = p.out[blockIdx.y];
    if (!out) return;
    const float* part = p.part + (int64_t)blockIdx.y * p.S * p.W;
    float v = 0.0f;
    if (col < p.W)
        for (int s = l; s < p.S; s += kSumRows) v += part[(int64_t)s * p.W + col];
    sm[l][c] = v;
    __syncthreads();
    for (int h = kSumRows / 2; h > 0; h /= 2) {
        if (l < h) sm[l][c] += sm[l + h][c];
        __syncthreads();
    }
    if (l == 0 && col < p.W) out[col] = sm[0][c];
}

template <typename F>
void for_types(const NormShape& s, F&& f) {
    if (s.io == SSM_F32) f(float(), float());
    else if (s.res == SSM_F32) f(bf16_t(), float());
    else f(bf16_t(), bf16_t());
}

}  // namespace

// A workgroup takes at least 4 rows a unit, and there are at most 1024 of
// them over all groups, so that the partial sums stay few beside the rows.
int norm_bwd_slices(const NormShape& s) {
    int upb = 1;
    for_row_shape(s.Wg, [&](auto rs) { upb = units_per_block<decltype(rs)::L>(); return 0; });
    const int64_t want = (s.M + 4 * (int64_t)upb - 1) / (4 * (int64_t)upb);
    const int64_t most = 1024 / s.G > 0 ? 1024 / s.G : 1;
    return (int)(want < 1 ? 1 : want < most ? want : most);
}

int launch_column_sums(const float* part, int S, int W, float* const out[3], int n_arr,
                       hipStream_t stream) {
    SumP p = {part, {out[0], out[1], out[2]}, S, W};
    column_sums<<<dim3((W + kSumCols - 1) / kSumCols, n_arr), kSumCols * kSumRows, 0, stream>>>(p);
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int launch_norm_residual_fwd(const ResidualArgs& a, hipStream_t stream) {
    const NormShape& s = a.s;
    FwdP p = {a.b, a.r, a.w_post, a.scale, a.w, a.r_out, a.h, a.rstd, a.rstd_post, a.r8, a.b8, a.h8,
              s.ld_x, s.ld_res, s.ld_out, s.M, s.scale_off, s.W, s.W32, s.eps, 1.0f / (float)s.W, s.alpha};
    if (!s.M) return SSM_OK;
    return for_row_shape(s.W, [&](auto rs) {
        using RS = decltype(rs);
        const dim3 grid = block_grid((s.M + units_per_block<RS::L>() - 1) / units_per_block<RS::L>());
        const int threads = row_threads<RS>(s.W);
        for_types(s, [&](auto t, auto r) {
            residual_fwd<decltype(t), decltype(r), RS::L, RS::NC><<<grid, threads, 0, stream>>>(p);
        });
        return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
    });
}

int launch_norm_residual_bwd(const ResidualBwdArgs& a, hipStream_t stream) {
    const NormShape& s = a.s;
    const int slices = norm_bwd_slices(s);
    const int64_t n = (int64_t)slices * s.W;
    auto part = [&](float* out, int i) { return !out ? nullptr : slices == 1 ? out : a.part + i * n; };
    BwdP p = {a.dh, a.dr_out, a.r_out, a.b, const_cast<uint8_t*>(a.r8), const_cast<uint8_t*>(a.b8),
              a.w_post, a.scale, a.w, a.rstd, a.rstd_post, a.d_r, a.d_b,
              part(a.d_w, 0), part(a.d_w_post, 1), part(a.d_scale, 2),
              s.ld_x, s.ld_res, s.ld_out, s.M, s.scale_off, s.W, s.W32, slices, 1.0f / (float)s.W, s.alpha};
    const int rc = for_row_shape(s.W, [&](auto rs) {
        using RS = decltype(rs);
        const int threads = row_threads<RS>(s.W);
        for_types(s, [&](auto t, auto r) {
            using T = decltype(t);
            using R = decltype(r);
            if (a.w_post || a.d_scale) residual_bwd<T, R, RS::L, RS::NC, true><<<slices, threads, 0, stream>>>(p);
            else residual_bwd<T, R, RS::L, RS::NC, false><<<slices, threads, 0, stream>>>(p);
        });
        return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
    });
    if (rc != SSM_OK || slices == 1 || !(a.d_w || a.d_w_post || a.d_scale)) return rc;
    float* const out[3] = {a.d_w, a.d_w_post, a.d_scale};
    return launch_column_sums(a.part, slices, s.W, out, a.d_w_post || a.d_scale ? 3 : 1, stream);
}

}  // namespace ssm
