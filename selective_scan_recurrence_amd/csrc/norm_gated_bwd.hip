// Backward of the gated norm (norm_gated.hip has the formulas): one pass over
// the rows, which gives d_y and d_z and, added up over a workgroup's rows in
// registers, a partial row of d_w; column_sums (norm_residual_bwd.hip) adds the
// partial rows.  Bound by HBM, and near it by the vector unit: about 30
// instructions a value, so idle lanes count (norm_rows.h, SEGMENTS: 16384 x
// 5120 in 8 groups of 640, 177 us with a wave of 64 lanes and two pieces for a
// group, 133 us with a workgroup a row).
#include "norm_gated.h"

namespace ssm {
namespace {

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

template <typename T, typename RS, Gate GATE, bool STREAM>
__global__ __launch_bounds__(RS::L ? kRowThreads : 1024) void gated_bwd(BwdP p) {
    constexpr int L = RS::L, NC = RS::NC, U = units_per_block<L>();
    constexpr Ends RAGGED = RS::RAGGED;
    // A workgroup's row with more than one piece a lane (groups past 8192) does
    // not fit the 128 registers that 1024 lanes leave each: none is loaded a row
    // ahead, each is loaded when it is needed, the second time from the caches.
    // 8192 x 16384 bf16: 1160 us with every piece held and half of them spilled,
    // 700 us so; 8192 x 12288: 920 and 605.  What bounds it now are spills still:
    // a lane past the end loads nothing and so keeps its piece, which makes every
    // piece live across the sum (gated: 28 to 56 registers spilled with two
    // pieces, 152 to 321 with four), beside the 16 or 32 column sums.
    constexpr bool LEAN = L == 0 && NC > 1;
    __shared__ SumMemory<L, NC, RS::SEGMENTS> lds;
    __shared__ float sm[L ? kRowThreads * 8 : 1];
    const RowLane<RS> lane(p.G, p.Wg);
    const Groups groups{p.G, p.Wg / 8};
    const int n = lane.n, c0 = lane.c0;
    struct Row {
        Piece<T> d[NC];
        PieceOr8<T> y[NC], z[NC];
        float rstd[NC];
    };
    int64_t row = (int64_t)lane.slice(p.G) * U + lane.ul.unit;
    const int64_t stride = (int64_t)p.slices * U;
    RowPtr<T> dout(p.dout, p.ld_out, row, c0), y(p.y, p.ld_y, row, c0), z(p.z, p.ld_z, row, c0);
    RowPtr<T> d_y(p.d_y, p.ld_y, row, c0), d_z(p.d_z, p.ld_z, row, c0);
    CkptRow y8(p.y8, p.scale_off, p.W32, row, c0), z8(p.z8, p.scale_off, p.W32, row, c0);
    RowPtr<float> rstd(p.rstd, p.G, row, 0);
    auto load_piece = [&](Row& r, int k) {
        const int at = lane.at(k);
        load8<RAGGED>(r.d[k], dout.p, at, n);
        if (!p.y8) load8<RAGGED>(r.y[k].t, y.p, at, n);
        else if (at < n) r.y[k].c = y8.load(at);
        r.rstd[k] = k == 0 || RS::SEGMENTS ? rstd.p[lane.group[k]] : r.rstd[0];
        if (GATE == kNone) return;
        if (!p.z8) load8<RAGGED>(r.z[k].t, z.p, at, n);
        else if (at < n) r.z[k].c = z8.load(at);
    };
    auto load = [&](Row& r) {
        if (LEAN) return;
#pragma unroll
        for (int k = 0; k < NC; ++k) load_piece(r, k);
    };
    auto skip_inputs = [&] {
        dout.skip(stride);
        y.skip(stride);
        z.skip(stride);
        y8.skip(stride);
        z8.skip(stride);
        rstd.skip(stride);
    };
    Row next;
    __builtin_memset(&next, 0, sizeof next);
    Piece<float> w[NC] = {};
    float dw[NC][8];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        if (!LEAN) fetch8<RAGGED>(w[k], p.w + c0, lane.at(k), n);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[k][j] = 0.0f;
    }
    lds.init();
    if (row < p.M) load(next);
    int turn = 0;
    walk_rows(next, row - lane.ul.unit, p.M, stride, [&](Row& r, Row& next) {
        if (!LEAN) {
            skip_inputs();
            if (row + stride < p.M) load(next);
        }
        const bool valid = row < p.M;  // else r is an earlier row: it is not counted again
        // x: the normalised value; yv, zv: y and z
        float x[NC][8], yv[NC][8], zv[NC][8], dot[NC], c1[NC];
        auto ready = [&](int k) {
            if (LEAN) {
                __builtin_amdgcn_sched_barrier(0);  // one piece at a time
                load_piece(r, k);
                fetch8<RAGGED>(w[k], p.w + c0, lane.at(k), n);
            }
            settle8<RAGGED>(r.d[k], lane.at(k), n);
            r.y[k].template values<RAGGED>(p.y8, yv[k], lane.at(k), n);
            if (GATE != kNone) r.z[k].template values<RAGGED>(p.z8, zv[k], lane.at(k), n);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[k][j] = (GATE == kBefore ? yv[k][j] * silu(zv[k][j]) : yv[k][j]) * r.rstd[k];
        };
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            ready(k);
            dot[k] = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float gate = GATE == kAfter ? silu(zv[k][j]) : 1.0f;
                const float dx = (GATE == kAfter ? r.d[k][j] * gate : r.d[k][j]) * x[k][j];
                if (valid) dw[k][j] += dx;
                dot[k] += dx * w[k][j];
            }
        }
        unit_sum(dot, c1, lds, turn++, lane.group, groups);
        if (valid) {
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                float dy[8], dz[8];
                if (LEAN) ready(k);
                c1[k] *= p.inv_n;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float s = GATE == kNone ? 0.0f : sigmoid(zv[k][j]);
                    const float gate = GATE == kNone ? 1.0f : zv[k][j] * s, slope = s * (1.0f + zv[k][j] * (1.0f - s));
                    const float dn = r.d[k][j] * w[k][j];
                    if (GATE == kAfter) {
                        dy[j] = r.rstd[k] * (dn * gate - x[k][j] * c1[k]);
                        dz[j] = dn * x[k][j] * slope;
                    } else {
                        const float du = r.rstd[k] * (dn - x[k][j] * c1[k]);
                        dy[j] = du * gate;
                        dz[j] = du * yv[k][j] * slope;
                    }
                }
                if (p.d_y) store8<RAGGED, STREAM>(d_y.p, lane.at(k), n, dy);
                if (GATE != kNone && p.d_z) store8<RAGGED, STREAM>(d_z.p, lane.at(k), n, dz);
            }
        }
        row += stride;
        if (LEAN) skip_inputs();
        d_y.skip(stride);
        d_z.skip(stride);
    });
    if (p.part) store_column_sums<L, NC, RAGGED>(p.part + (int64_t)lane.slice(p.G) * p.W + c0, n, dw, sm);
}

}  // namespace

int launch_norm_gated_bwd(const GatedBwdArgs& a, hipStream_t stream) {
    const NormShape& s = a.s;
    const int slices = norm_bwd_slices(s, true);
    BwdP p = {a.dout, a.y, a.z, const_cast<uint8_t*>(a.y8), const_cast<uint8_t*>(a.z8), a.w, a.rstd,
              a.d_y, a.d_z, a.d_w ? (slices == 1 ? a.d_w : a.part) : nullptr, s.ld_x, s.ld_z,
              s.ld_out, s.M, s.scale_off, s.G, s.W, s.Wg, s.W32, slices, 1.0f / (float)s.Wg};
    const int rc = for_row_shape<kGatedBwd>(s.M, s.W, s.G, [&](auto rs, int threads, int units) {
        using RS = decltype(rs);
        const unsigned grid = (unsigned)(slices * units);
        for_gate<RS>(s, a.z || a.z8, 5, [&](auto t, auto gate, auto past) {
            gated_bwd<decltype(t), RS, gate.value, past.value><<<grid, threads, 0, stream>>>(p);
        });
        return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
    });
    if (rc != SSM_OK || !a.d_w || slices == 1) return rc;
    return launch_column_sums(a.part, slices, s.W, ColumnSums{a.d_w}, stream);
}

}  // namespace ssm
