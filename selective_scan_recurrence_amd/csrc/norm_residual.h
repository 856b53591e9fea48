// What the residual norm's two directions share (norm_residual.hip has the
// formulas).
#pragma once

#include "block_internal.h"
#include "norm_rows.h"

namespace ssm {

// e of this lane's pieces
template <Ends RAGGED>
__device__ __forceinline__ Piece<float> branch_factor(const float* w_post, const float* scale, float alpha, int at, int n) {
    Piece<float> e = {}, t = {};
#pragma unroll
    for (int j = 0; j < 8; ++j) e.d[j] = alpha;
    if (scale) {
        fetch8<RAGGED>(t, scale, at, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) e.d[j] *= t.d[j];
    }
    if (w_post) {
        fetch8<RAGGED>(t, w_post, at, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) e.d[j] *= t.d[j];
    }
    return e;
}

// Host: calls f(io element, residual element).
template <typename F>
void for_types(const NormShape& s, F&& f) {
    if (s.io == SSM_F32) f(float(), float());
    else if (s.res == SSM_F32) f(bf16_t(), float());
    else f(bf16_t(), bf16_t());
}

}  // namespace ssm
