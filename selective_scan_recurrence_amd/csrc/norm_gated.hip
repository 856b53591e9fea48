// The gated norm after the scan, forward and backward.  Per row and group:
//   gate before:  u = y SiLU(z),  out = u rstd w,  rstd = 1 / sqrt(mean u^2 + eps)
//   gate after:   out = y rstd w SiLU(z),          rstd from y
// and, with c() the mean over the group, s = sigmoid(z), g' = s (1 + z (1 - s)):
//   before:  x = u rstd, dn = dout w, du = rstd (dn - x c(dn x)),
//            dy = du SiLU(z), dz = du y g', dw = sum_rows dout x
//   after:   x = y rstd, dn = dout SiLU(z) w, dy = rstd (dn - x c(dn x)),
//            dz = dout x w g', dw = sum_rows dout SiLU(z) x
// All of it in f32; what is stored in bf16 is rounded once.
//
// Bound by HBM: each input is read once and each output written once, the
// group held in registers between the sum and the outputs (norm_rows.h).
#include "block_internal.h"
#include "norm_rows.h"

namespace ssm {
namespace {

enum Gate { kNone, kBefore, kAfter };

struct FwdP {
    const void *y, *z;
    const float* w;
    void* out;
    float* rstd;
    uint8_t *y8, *z8, *out8;
    int64_t ld_y, ld_z, ld_out, M, scale_off;
    int G, Wg, W32, slices;
    float eps, inv_n;
};

// Workgroup (slice, group) takes every slices-th row (or set of rows), and
// loads the next one while it works on the present one.  w stays in registers:
// a load between the next row's and their use would have to wait for them.
template <typename T, int L, int NC, bool RAGGED, Gate GATE>
__global__ __launch_bounds__(L ? kRowThreads : 1024) void gated_fwd(FwdP p) {
    __shared__ float lds[32];
    constexpr int U = units_per_block<L>();
    const UnitLane ul = unit_lane<L>();
    const int g = blockIdx.x % p.G, c0 = g * p.Wg, wg = p.Wg;
    const T* y = static_cast<const T*>(p.y) + c0;
    const T* z = static_cast<const T*>(p.z) + c0;
    T* out = static_cast<T*>(p.out) + c0;
    const Ckpt y8(p.y8, p.scale_off, p.W32, c0), z8(p.z8, p.scale_off, p.W32, c0), out8(p.out8, p.scale_off, p.W32, c0);
    struct Row {
        Piece<T> y[NC], z[NC];
    };
    auto load = [&](Row& r, int64_t row) {
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            load8<RAGGED>(r.y[k], y + row * p.ld_y, ul.at(k), wg);
            if (GATE != kNone) load8<RAGGED>(r.z[k], z + row * p.ld_z, ul.at(k), wg);
        }
    };
    // lanes past the width keep the zeros they start with
    Row next = {};
    Piece<float> w[NC] = {};
#pragma unroll
    for (int k = 0; k < NC; ++k) load8<RAGGED>(w[k], p.w + c0, ul.at(k), wg);
    unit_sum_init<L>(lds);
    int64_t row = (int64_t)(blockIdx.x / p.G) * U + ul.unit;
    const int64_t step = (int64_t)p.slices * U;
    if (row < p.M) load(next, row);
    int turn = 0;
    for (int64_t first = row - ul.unit; first < p.M; first += step, row += step, ++turn) {
        const Row r = next;
        if (row + step < p.M) load(next, row + step);
        float x[NC][8], ss = 0.0f;  // x: what is normalised
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[k][j] = GATE == kBefore ? r.y[k][j] * silu(r.z[k][j]) : r.y[k][j];
                ss += x[k][j] * x[k][j];
            }
        const float rstd = rsqrt1(unit_sum<L>(ss, lds, turn) * p.inv_n + p.eps);
        if (row >= p.M) continue;
        if (p.rstd && ul.lane == 0) p.rstd[row * p.G + g] = rstd;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                o[j] = x[k][j] * rstd * w[k][j];
                if (GATE == kAfter) o[j] *= silu(r.z[k][j]);
            }
            store8<RAGGED>(out + row * p.ld_out, ul.at(k), wg, o);
            if (ul.at(k) >= (wg + 31) / 32 * 32) continue;
            float v[8];
            if (p.y8) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = r.y[k][j];
                y8.store(row, ul.at(k), v);
            }
            if (GATE != kNone && p.z8) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = r.z[k][j];
                z8.store(row, ul.at(k), v);
            }
            if (p.out8) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = as_stored(o[j], T());
                out8.store(row, ul.at(k), v);
            }
        }
    }
}

struct BwdP {
    const void *dout, *y, *z;
    uint8_t *y8, *z8;
    const float *w, *rstd;
    void *d_y, *d_z;
    float* part;  // [slices][W], or null without d_w
    int64_t ld_y, ld_z, ld_out, M, scale_off;
    int G, W, Wg, W32, slices;
    float inv_n;
};

template <typename T, int L, int NC, bool RAGGED, Gate GATE>
__global__ __launch_bounds__(L ? kRowThreads : 1024) void gated_bwd(BwdP p) {
    __shared__ float lds[L ? kRowThreads * 8 : 32];
    constexpr int U = units_per_block<L>();
    const UnitLane ul = unit_lane<L>();
    const int g = blockIdx.x % p.G, slice = blockIdx.x / p.G, c0 = g * p.Wg, wg = p.Wg;
    const T* dout = static_cast<const T*>(p.dout) + c0;
    const T* y = static_cast<const T*>(p.y) + c0;
    const T* z = static_cast<const T*>(p.z) + c0;
    T* d_y = static_cast<T*>(p.d_y) + c0;
    T* d_z = static_cast<T*>(p.d_z) + c0;
    const Ckpt y8(p.y8, p.scale_off, p.W32, c0), z8(p.z8, p.scale_off, p.W32, c0);
    struct Row {
        Piece<T> d[NC];
        PieceOr8<T> y[NC], z[NC];
        float rstd;
    };
    auto load = [&](Row& r, int64_t row) {
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            load8<RAGGED>(r.d[k], dout + row * p.ld_out, ul.at(k), wg);
            if (!p.y8) load8<RAGGED>(r.y[k].t, y + row * p.ld_y, ul.at(k), wg);
            else if (ul.at(k) < wg) r.y[k].c = y8.load(row, ul.at(k));
            if (GATE == kNone) continue;
            if (!p.z8) load8<RAGGED>(r.z[k].t, z + row * p.ld_z, ul.at(k), wg);
            else if (ul.at(k) < wg) r.z[k].c = z8.load(row, ul.at(k));
        }
        r.rstd = p.rstd[row * p.G + g];
    };
    Row next;
    __builtin_memset(&next, 0, sizeof next);
    Piece<float> w[NC] = {};
    float dw[NC][8];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        load8<RAGGED>(w[k], p.w + c0, ul.at(k), wg);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[k][j] = 0.0f;
    }
    unit_sum_init<L>(lds);
    int64_t row = (int64_t)slice * U + ul.unit;
    const int64_t step = (int64_t)p.slices * U;
    if (row < p.M) load(next, row);
    int turn = 0;
    for (int64_t first = row - ul.unit; first < p.M; first += step, row += step, ++turn) {
        const Row r = next;
        if (row + step < p.M) load(next, row + step);
        const bool valid = row < p.M;  // else r is the row before: it is not counted again
        // x: the normalised value; yv, zv: y and z
        float x[NC][8], yv[NC][8], zv[NC][8], dot = 0.0f;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            if (p.y8) r.y[k].c.values(yv[k]);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) yv[k][j] = r.y[k].t[j];
            if (GATE != kNone) {
                if (p.z8) r.z[k].c.values(zv[k]);
                else
#pragma unroll
                    for (int j = 0; j < 8; ++j) zv[k][j] = r.z[k].t[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float gate = GATE == kNone ? 1.0f : silu(zv[k][j]);
                x[k][j] = (GATE == kBefore ? yv[k][j] * gate : yv[k][j]) * r.rstd;
                const float dx = (GATE == kAfter ? r.d[k][j] * gate : r.d[k][j]) * x[k][j];
                if (valid) dw[k][j] += dx;
                dot += dx * w[k][j];
            }
        }
        const float c1 = unit_sum<L>(dot, lds, turn) * p.inv_n;
        if (!valid) continue;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            float dy[8], dz[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float s = GATE == kNone ? 0.0f : sigmoid(zv[k][j]);
                const float gate = GATE == kNone ? 1.0f : zv[k][j] * s, slope = s * (1.0f + zv[k][j] * (1.0f - s));
                const float dn = r.d[k][j] * w[k][j];
                if (GATE == kAfter) {
                    dy[j] = r.rstd * (dn * gate - x[k][j] * c1);
                    dz[j] = dn * x[k][j] * slope;
                } else {
                    const float du = r.rstd * (dn - x[k][j] * c1);
                    dy[j] = du * gate;
                    dz[j] = du * yv[k][j] * slope;
                }
            }
            if (p.d_y) store8<RAGGED>(d_y + row * p.ld_y, ul.at(k), wg, dy);
            if (GATE != kNone && p.d_z) store8<RAGGED>(d_z + row * p.ld_z, ul.at(k), wg, dz);
        }
    }
    if (p.part) store_column_sums<L, NC, RAGGED>(p.part + (int64_t)slice * p.W + c0, wg, dw, lds);
}

}  // namespace

int launch_norm_gated_fwd(const GatedArgs& a, hipStream_t stream) {
    const NormShape& s = a.s;
    if (!s.M) return SSM_OK;
    return for_row_shape(s.Wg, [&](auto rs) {
        using RS = decltype(rs);
        const int threads = row_threads<RS>(s.Wg), slices = row_slices<RS>(s.M, s.G, threads);
        FwdP p = {a.y, a.z, a.w, a.out, a.rstd, a.y8, a.z8, a.out8, s.ld_x, s.ld_z, s.ld_out,
                  s.M, s.scale_off, s.G, s.Wg, s.W32, slices, s.eps, 1.0f / (float)s.Wg};
        const unsigned grid = (unsigned)(slices * s.G);
        auto go = [&](auto t) {
            using T = decltype(t);
            if (!a.z) gated_fwd<T, RS::L, RS::NC, RS::RAGGED, kNone><<<grid, threads, 0, stream>>>(p);
            else if (s.after) gated_fwd<T, RS::L, RS::NC, RS::RAGGED, kAfter><<<grid, threads, 0, stream>>>(p);
            else gated_fwd<T, RS::L, RS::NC, RS::RAGGED, kBefore><<<grid, threads, 0, stream>>>(p);
        };
        if (s.io == SSM_BF16) go(bf16_t());
        else go(float());
        return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
    });
}

int launch_norm_gated_bwd(const GatedBwdArgs& a, hipStream_t stream) {
    const NormShape& s = a.s;
    const int slices = norm_bwd_slices(s);
    BwdP p = {a.dout, a.y, a.z, const_cast<uint8_t*>(a.y8), const_cast<uint8_t*>(a.z8), a.w, a.rstd,
              a.d_y, a.d_z, a.d_w ? (slices == 1 ? a.d_w : a.part) : nullptr, s.ld_x, s.ld_z,
              s.ld_out, s.M, s.scale_off, s.G, s.W, s.Wg, s.W32, slices, 1.0f / (float)s.Wg};
    const int rc = for_row_shape(s.Wg, [&](auto rs) {
        using RS = decltype(rs);
        const int threads = row_threads<RS>(s.Wg);
        const unsigned grid = (unsigned)(slices * s.G);
        auto go = [&](auto t) {
            using T = decltype(t);
            if (!a.z && !a.z8) gated_bwd<T, RS::L, RS::NC, RS::RAGGED, kNone><<<grid, threads, 0, stream>>>(p);
            else if (s.after) gated_bwd<T, RS::L, RS::NC, RS::RAGGED, kAfter><<<grid, threads, 0, stream>>>(p);
            else gated_bwd<T, RS::L, RS::NC, RS::RAGGED, kBefore><<<grid, threads, 0, stream>>>(p);
        };
        if (s.io == SSM_BF16) go(bf16_t());
        else go(float());
        return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
    });
    if (rc != SSM_OK || !a.d_w || slices == 1) return rc;
    return launch_column_sums(a.part, slices, s.W, ColumnSums{a.d_w}, stream);
}

}  // namespace ssm
