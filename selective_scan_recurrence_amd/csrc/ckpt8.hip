// Writing a tensor as its 8-bit checkpoint and reading one back (ckpt8.h has
// the format).  A lane takes 8 consecutive values; four lanes share a block.
// Bound by HBM: the values cross it once in their type and once in 33/32
// bytes.
#include "block_internal.h"
#include "norm_rows.h"

namespace ssm {
namespace {

template <typename T>
__global__ __launch_bounds__(256) void ckpt8_pack(const T* __restrict__ x, int64_t ld, uint8_t* out,
                                                  int64_t pieces, int P, int W, int W32, int64_t scale_off) {
    const int64_t i = block_id() * 256 + threadIdx.x;
    if (i >= pieces) return;  // pieces is a multiple of 4: a block's lanes go together
    const int64_t row = i / P;
    const int at = 8 * (int)(i % P);
    Piece<T> t = {};
    load8<true>(t, x + row * ld, at, W);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = t[j];
    Ckpt(out, scale_off, W32, 0).store(row, at, v);
}

template <typename T>
__global__ __launch_bounds__(256) void ckpt8_unpack(uint8_t* x8, T* __restrict__ x, int64_t ld,
                                                    int64_t pieces, int P, int W, int W32, int64_t scale_off) {
    const int64_t i = block_id() * 256 + threadIdx.x;
    if (i >= pieces) return;
    const int64_t row = i / P;
    const int at = 8 * (int)(i % P);
    if (at >= W) return;
    float v[8];
    Ckpt(x8, scale_off, W32, 0).load(row, at).values(v);
    store8<true>(x + row * ld, at, W, v);
}

}  // namespace

int launch_ckpt8_pack(const void* x, int64_t ld, int64_t M, int64_t W, int dtype, uint8_t* out,
                      hipStream_t stream) {
    const int64_t W32 = ckpt8_width(W), pieces = M * (W32 / 8);
    if (!pieces) return SSM_OK;
    const dim3 grid = block_grid((pieces + 255) / 256);
    if (dtype == SSM_BF16)
        ckpt8_pack<bf16_t><<<grid, 256, 0, stream>>>(static_cast<const bf16_t*>(x), ld, out, pieces,
                                                     (int)(W32 / 8), (int)W, (int)W32, M * W32);
    else
        ckpt8_pack<float><<<grid, 256, 0, stream>>>(static_cast<const float*>(x), ld, out, pieces,
                                                    (int)(W32 / 8), (int)W, (int)W32, M * W32);
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int launch_ckpt8_unpack(const uint8_t* x8, void* x, int64_t ld, int64_t M, int64_t W, int dtype,
                        hipStream_t stream) {
    const int64_t W32 = ckpt8_width(W), pieces = M * (W32 / 8);
    if (!pieces) return SSM_OK;
    const dim3 grid = block_grid((pieces + 255) / 256);
    uint8_t* in = const_cast<uint8_t*>(x8);
    if (dtype == SSM_BF16)
        ckpt8_unpack<bf16_t><<<grid, 256, 0, stream>>>(in, static_cast<bf16_t*>(x), ld, pieces,
                                                       (int)(W32 / 8), (int)W, (int)W32, M * W32);
    else
        ckpt8_unpack<float><<<grid, 256, 0, stream>>>(in, static_cast<float*>(x), ld, pieces,
                                                      (int)(W32 / 8), (int)W, (int)W32, M * W32);
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // namespace ssm
