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
#include "norm_gated.h"

namespace ssm {
namespace {

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
template <typename T, typename RS, Gate GATE, bool STREAM>
__global__ __launch_bounds__(RS::L ? kRowThreads : 1024) void gated_fwd(FwdP p) {
    constexpr int L = RS::L, NC = RS::NC, U = units_per_block<L>();
    constexpr Ends RAGGED = RS::RAGGED;
    __shared__ SumMemory<L, NC, RS::SEGMENTS> lds;
    const RowLane<RS> lane(p.G, p.Wg);
    const Groups groups{p.G, p.Wg / 8};
    const int n = lane.n, c0 = lane.c0;
    struct Row {
        Piece<T> y[NC], z[NC];
    };
    int64_t row = (int64_t)lane.slice(p.G) * U + lane.ul.unit;
    const int64_t stride = (int64_t)p.slices * U;
    RowPtr<T> y(p.y, p.ld_y, row, c0), z(p.z, p.ld_z, row, c0), out(p.out, p.ld_out, row, c0);
    CkptRow y8(p.y8, p.scale_off, p.W32, row, c0), z8(p.z8, p.scale_off, p.W32, row, c0);
    CkptRow out8(p.out8, p.scale_off, p.W32, row, c0);
    auto load = [&](Row& r) {
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            load8<RAGGED>(r.y[k], y.p, lane.at(k), n);
            if (GATE != kNone) load8<RAGGED>(r.z[k], z.p, lane.at(k), n);
        }
    };
    // lanes past the width keep the zeros they start with
    Row next = {};
    Piece<float> w[NC] = {};
#pragma unroll
    for (int k = 0; k < NC; ++k) fetch8<RAGGED>(w[k], p.w + c0, lane.at(k), n);
    lds.init();
    if (row < p.M) load(next);
    int turn = 0;
    walk_rows(next, row - lane.ul.unit, p.M, stride, [&](Row& r, Row& next) {
        y.skip(stride);
        z.skip(stride);
        if (row + stride < p.M) load(next);
        float x[NC][8], ss[NC], rstd[NC];  // x: what is normalised
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            settle8<RAGGED>(r.y[k], lane.at(k), n);
            if (GATE != kNone) settle8<RAGGED>(r.z[k], lane.at(k), n);
            ss[k] = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[k][j] = GATE == kBefore ? r.y[k][j] * silu(r.z[k][j]) : r.y[k][j];
                ss[k] += x[k][j] * x[k][j];
            }
        }
        unit_rstd(ss, [&](int k, int j) { return x[k][j]; }, rstd, lds, turn, lane.group, groups, p.inv_n, p.eps);
        if (row < p.M) {
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                const int at = lane.at(k);
                if (p.rstd && (RS::SEGMENTS ? at < n && at % p.Wg == 0 : at == 0)) p.rstd[row * p.G + lane.group[k]] = rstd[k];
                float o[8], v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    o[j] = x[k][j] * rstd[k] * w[k][j];
                    if (GATE == kAfter) o[j] *= silu(r.z[k][j]);
                }
                store8<RAGGED, STREAM>(out.p, at, n, o);
                if (at >= (n + 31) / 32 * 32) continue;
                if (p.y8) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = r.y[k][j];
                    y8.store(at, v);
                }
                if (GATE != kNone && p.z8) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = r.z[k][j];
                    z8.store(at, v);
                }
                if (p.out8) {
                    as_stored<T>(o, v);
                    out8.store(at, v);
                }
            }
        }
        row += stride;
        out.skip(stride);
        y8.skip(stride);
        z8.skip(stride);
        out8.skip(stride);
    });
}

}  // namespace

int launch_norm_gated_fwd(const GatedArgs& a, hipStream_t stream) {
    const NormShape& s = a.s;
    if (!s.M) return SSM_OK;
    return for_row_shape<kGatedFwd>(s.M, s.W, s.G, [&](auto rs, int threads, int units) {
        using RS = decltype(rs);
        const int slices = row_slices<RS>(s.M, units, threads);
        FwdP p = {a.y, a.z, a.w, a.out, a.rstd, a.y8, a.z8, a.out8, s.ld_x, s.ld_z, s.ld_out,
                  s.M, s.scale_off, s.G, s.Wg, s.W32, slices, s.eps, 1.0f / (float)s.Wg};
        const unsigned grid = (unsigned)(slices * units);
        for_gate<RS>(s, a.z, 3, [&](auto t, auto gate, auto past) {
            gated_fwd<decltype(t), RS, gate.value, past.value><<<grid, threads, 0, stream>>>(p);
        });
        return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
    });
}

}  // namespace ssm
