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

struct FwdP {
    const void *y, *z;
    const float* w;
    void* out;
    float* rstd;
    uint8_t *y8, *z8, *out8;
    int64_t ld_y, ld_z, ld_out, units, scale_off;
    int G, Wg, W32;
    float eps, inv_n;
};

template <typename T, int L, int NC, bool AFTER>
__global__ __launch_bounds__(L ? kRowThreads : 1024) void gated_fwd(FwdP p) {
    __shared__ float lds[32];
    const UnitLane ul = unit_lane<L>();
    const int64_t id = block_id() * units_per_block<L>() + ul.unit;
    const bool valid = id < p.units;
    const int64_t row = valid ? id / p.G : 0;
    const int g = valid ? (int)(id % p.G) : 0, c0 = g * p.Wg;
    const int wg = valid ? p.Wg : 0;
    const T* y = static_cast<const T*>(p.y) + row * p.ld_y + c0;
    const T* z = p.z ? static_cast<const T*>(p.z) + row * p.ld_z + c0 : nullptr;
    Piece<T> yv[NC], zv[NC];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = ul.lane + k * ul.lanes, n = wg - 8 * c;
        if (n > 0) {
            yv[k] = load8(y + 8 * c, n);
            if (z) zv[k] = load8(z + 8 * c, n);
        }
    }
    // x: what is normalised; ga: the gate after the norm
    float x[NC][8], ga[NC][8], ss = 0.0f;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const bool on = wg - 8 * (ul.lane + k * ul.lanes) > 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float yj = on ? yv[k][j] : 0.0f, gj = !on ? 0.0f : z ? silu(zv[k][j]) : 1.0f;
            x[k][j] = AFTER ? yj : yj * gj;
            ga[k][j] = AFTER ? gj : 1.0f;
            ss += x[k][j] * x[k][j];
        }
    }
    const float rstd = 1.0f / sqrtf(unit_sum<L>(ss, lds, 0) * p.inv_n + p.eps);
    if (valid && p.rstd && ul.lane == 0) p.rstd[id] = rstd;
    T* out = static_cast<T*>(p.out) + row * p.ld_out + c0;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = ul.lane + k * ul.lanes, n = wg - 8 * c;
        float o[8] = {};
        if (n > 0) {
            const Piece<float> w = load8(p.w + c0 + 8 * c, n);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = x[k][j] * rstd * w[j] * ga[k][j];
            store8(out + 8 * c, n, o);
        }
        if (8 * c < (valid ? (wg + 31) / 32 * 32 : 0)) {
            float v[8];
            if (p.y8) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = n > 0 ? yv[k][j] : 0.0f;
                ckpt_store(ckpt_row(p.y8, p.scale_off, p.W32, row, c0), c, v);
            }
            if (p.z8) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = n > 0 ? zv[k][j] : 0.0f;
                ckpt_store(ckpt_row(p.z8, p.scale_off, p.W32, row, c0), c, v);
            }
            if (p.out8) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = as_stored(o[j], T());
                ckpt_store(ckpt_row(p.out8, p.scale_off, p.W32, row, c0), c, v);
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

template <typename T, int L, int NC, bool AFTER>
__global__ __launch_bounds__(L ? kRowThreads : 1024) void gated_bwd(BwdP p) {
    __shared__ float lds[L ? kRowThreads * 8 : 32];
    const UnitLane ul = unit_lane<L>();
    const int g = blockIdx.x % p.G, slice = blockIdx.x / p.G, c0 = g * p.Wg;
    const bool gate = p.z || p.z8;
    float w[NC][8], dw[NC][8];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = ul.lane + k * ul.lanes, n = p.Wg - 8 * c;
        if (n > 0) {
            const Piece<float> t = load8(p.w + c0 + 8 * c, n);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[k][j] = t[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (n <= 0) w[k][j] = 0.0f;
            dw[k][j] = 0.0f;
        }
    }
    int turn = 0;
    const int64_t step = (int64_t)p.slices * units_per_block<L>();
    for (int64_t r0 = (int64_t)slice * units_per_block<L>(); r0 < p.M; r0 += step, ++turn) {
        const int64_t row = r0 + ul.unit;
        const bool valid = row < p.M;
        const int wg = valid ? p.Wg : 0;
        const int64_t rr = valid ? row : 0;
        const float rstd = valid ? p.rstd[rr * p.G + g] : 0.0f;
        // d: dout; x: the normalised value; then what dy and dz need
        float d[NC][8], x[NC][8], y[NC][8], z[NC][8], dot = 0.0f;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int c = ul.lane + k * ul.lanes, n = wg - 8 * c;
#pragma unroll
            for (int j = 0; j < 8; ++j) d[k][j] = y[k][j] = z[k][j] = 0.0f;
            if (n > 0) {
                const Piece<T> t = load8(static_cast<const T*>(p.dout) + rr * p.ld_out + c0 + 8 * c, n);
#pragma unroll
                for (int j = 0; j < 8; ++j) d[k][j] = t[j];
                if (p.y8) {
                    ckpt_load(ckpt_row(p.y8, p.scale_off, p.W32, rr, c0), c, y[k]);
                } else {
                    const Piece<T> u = load8(static_cast<const T*>(p.y) + rr * p.ld_y + c0 + 8 * c, n);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[k][j] = u[j];
                }
                if (p.z8) {
                    ckpt_load(ckpt_row(p.z8, p.scale_off, p.W32, rr, c0), c, z[k]);
                } else if (gate) {
                    const Piece<T> u = load8(static_cast<const T*>(p.z) + rr * p.ld_z + c0 + 8 * c, n);
#pragma unroll
                    for (int j = 0; j < 8; ++j) z[k][j] = u[j];
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float gj = gate ? silu(z[k][j]) : 1.0f;
                x[k][j] = (AFTER ? y[k][j] : y[k][j] * gj) * rstd;
                const float dn = AFTER ? d[k][j] * gj : d[k][j];
                if (n > 0) dw[k][j] += dn * x[k][j];
                dot += dn * w[k][j] * x[k][j];
            }
        }
        const float c1 = unit_sum<L>(dot, lds, turn) * p.inv_n;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int c = ul.lane + k * ul.lanes, n = wg - 8 * c;
            if (n <= 0) continue;
            float dy[8], dz[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float sg = sigmoid(z[k][j]);
                const float gj = gate ? z[k][j] * sg : 1.0f, slope = sg * (1.0f + z[k][j] * (1.0f - sg));
                if (AFTER) {
                    dy[j] = rstd * (d[k][j] * gj * w[k][j] - x[k][j] * c1);
                    dz[j] = d[k][j] * x[k][j] * w[k][j] * slope;
                } else {
                    const float du = rstd * (d[k][j] * w[k][j] - x[k][j] * c1);
                    dy[j] = du * gj;
                    dz[j] = du * y[k][j] * slope;
                }
            }
            if (p.d_y) store8(static_cast<T*>(p.d_y) + rr * p.ld_y + c0 + 8 * c, n, dy);
            if (p.d_z) store8(static_cast<T*>(p.d_z) + rr * p.ld_z + c0 + 8 * c, n, dz);
        }
    }
    if (p.part) store_column_sums<L, NC>(p.part + (int64_t)slice * p.W + c0, p.Wg, dw, lds);
}

}  // namespace

int launch_norm_gated_fwd(const GatedArgs& a, hipStream_t stream) {
    const NormShape& s = a.s;
    FwdP p = {a.y, a.z, a.w, a.out, a.rstd, a.y8, a.z8, a.out8, s.ld_x, s.ld_z, s.ld_out,
              s.M * s.G, s.scale_off, s.G, s.Wg, s.W32, s.eps, 1.0f / (float)s.Wg};
    if (!p.units) return SSM_OK;
    return for_row_shape(s.Wg, [&](auto rs) {
        using RS = decltype(rs);
        const dim3 grid = block_grid((p.units + units_per_block<RS::L>() - 1) / units_per_block<RS::L>());
        const int threads = row_threads<RS>(s.Wg);
        auto go = [&](auto t) {
            using T = decltype(t);
            if (s.after) gated_fwd<T, RS::L, RS::NC, true><<<grid, threads, 0, stream>>>(p);
            else gated_fwd<T, RS::L, RS::NC, false><<<grid, threads, 0, stream>>>(p);
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
            if (s.after) gated_bwd<T, RS::L, RS::NC, true><<<grid, threads, 0, stream>>>(p);
            else gated_bwd<T, RS::L, RS::NC, false><<<grid, threads, 0, stream>>>(p);
        };
        if (s.io == SSM_BF16) go(bf16_t());
        else go(float());
        return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
    });
    if (rc != SSM_OK || !a.d_w || slices == 1) return rc;
    float* const out[3] = {a.d_w, nullptr, nullptr};
    return launch_column_sums(a.part, slices, s.W, out, 1, stream);
}

}  // namespace ssm
