// Weight gradient of a projection whose input was kept as an 8-bit checkpoint:
//   dw[o][c] = sum_m dy[m][o] x[m][c] (+ dw[o][c]),  x = code * 2^k.
// A workgroup owns a 64 x 64 tile of dw and walks the rows 16 at a time.
#include "block_internal.h"
#include "norm_rows.h"

namespace ssm {
namespace {

constexpr int kT = 64, kK = 16;

template <typename T>
__global__ __launch_bounds__(256) void wgrad_tile(const T* __restrict__ dy, int64_t ld, const uint8_t* __restrict__ x8,
                                                  float* dw, int64_t M, int W, int W32, int O, int64_t scale_off,
                                                  bool accumulate) {
    __shared__ float a[kK][kT], b[kK][kT];
    const int o0 = blockIdx.y * kT, c0 = blockIdx.x * kT, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int64_t m0 = 0; m0 < M; m0 += kK) {
        for (int i = threadIdx.x; i < kK * kT; i += 256) {
            const int r = i / kT, e = i % kT;
            const int64_t m = m0 + r;
            a[r][e] = m < M && o0 + e < O ? to_f32(dy[m * ld + o0 + e]) : 0.0f;
            float v = 0.0f;
            if (m < M && c0 + e < W) {
                const uint8_t code = x8[m * W32 + c0 + e];
                const uint8_t s = x8[scale_off + m * (W32 / 32) + (c0 + e) / 32];
                v = __builtin_amdgcn_cvt_pk_f32_fp8((int)code, false)[0] * ckpt8_scale(s);
            }
            b[r][e] = v;
        }
        __syncthreads();
        for (int r = 0; r < kK; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += a[r][ty + 16 * i] * b[r][tx + 16 * j];
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int o = o0 + ty + 16 * i, c = c0 + tx + 16 * j;
            if (o < O && c < W) {
                float* p = dw + (int64_t)o * W + c;
                *p = accumulate ? *p + acc[i][j] : acc[i][j];
            }
        }
}

}  // namespace

size_t ckpt8_wgrad_workspace_bytes(int64_t, int64_t, int64_t, int) { return 0; }

int launch_ckpt8_wgrad(const void* dy, int64_t ld, const uint8_t* x8, float* dw, int64_t M, int64_t W,
                       int64_t O, int dtype, bool accumulate, void*, hipStream_t stream) {
    const dim3 grid((unsigned)((W + kT - 1) / kT), (unsigned)((O + kT - 1) / kT));
    const int64_t W32 = ckpt8_width(W);
    if (dtype == SSM_BF16)
        wgrad_tile<bf16_t><<<grid, 256, 0, stream>>>(static_cast<const bf16_t*>(dy), ld, x8, dw, M, (int)W,
                                                     (int)W32, (int)O, M * W32, accumulate);
    else
        wgrad_tile<float><<<grid, 256, 0, stream>>>(static_cast<const float*>(dy), ld, x8, dw, M, (int)W,
                                                    (int)W32, (int)O, M * W32, accumulate);
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // namespace ssm
