// How the weight gradient's rows are dealt to workgroups (ckpt8_wgrad.hip): a
// plan made on the host and read on the device, without either's headers, so
// that it can be checked for every size without a launch.
#pragma once

#include <stdint.h>

#include "ssm.h"

#ifdef __HIPCC__
#define SSM_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SSM_HOST_DEVICE inline
#endif

namespace ssm {

// A tile of dw, kTO x kTC, takes the rows in steps of kTM.
constexpr int kTO = 256, kTC = 128, kTM = 64;

// count parts of the rows; part i starts at row i * rows, a multiple of kTM.
struct RowSplit {
    int count, rows;
};

// One past the last of part i's rows.  The last part's whole length may pass
// both M and the largest int, so the end is not formed from it.
SSM_HOST_DEVICE int part_end(int M, int rows, int i) {
    const int begin = i * rows;
    return M - begin < rows ? M : begin + rows;
}

// Parts of the rows, each of at least a step: the count with the least
// modelled time.  A step takes 1.25 us with one workgroup on a compute unit
// and 2.0 with two (bf16), 3.9 with the one that f32 has room for; the join
// costs a launch and moves each partial twice at 5 TB/s.  (8192 x 1024 x 512
// in bf16, 16 tiles: 36 us with the 32 parts that fill the chip, 24 with 10.)
inline RowSplit split_rows(int64_t M, int64_t W, int64_t O, int dtype) {
    const int64_t tiles = ((W + kTC - 1) / kTC) * ((O + kTO - 1) / kTO), steps = (M + kTM - 1) / kTM;
    RowSplit best{1, (int)((steps ? steps : 1) * kTM)};
    double best_us = 0;
    for (int64_t n = 1, next; n == 1 || (n <= steps && n * tiles <= 512); n = next) {
        const int64_t each = steps ? (steps + n - 1) / n : 1, count = steps ? (steps + each - 1) / each : 1;
        const int64_t wgs = tiles * count, left = wgs % 512;
        const double step_us = dtype == SSM_BF16 ? (double)(wgs / 512) * 2.0 + (left == 0 ? 0.0 : left <= 256 ? 1.25 : 2.0)
                                                 : (double)((wgs + 255) / 256) * 3.9;
        const double us = step_us * (double)each + (count > 1 ? 4.0 + (double)count * W * O * 8.0 / 5e6 : 0.0);
        if (n == 1 || us < best_us) {
            best = RowSplit{(int)count, (int)(each * kTM)};
            best_us = us;
        }
        next = each > 1 ? (steps + each - 2) / (each - 1) : n + steps + 1;  // the next count with fewer steps each
    }
    return best;
}

}  // namespace ssm
