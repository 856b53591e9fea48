// Writing a tensor as its 8-bit checkpoint and reading one back (ckpt8.h has
// the format).  A lane takes 8 consecutive values; four lanes share a block.
// Bound by HBM: the values cross it once in their type and once in 33/32
// bytes.
#include <type_traits>

#include "block_internal.h"
#include "norm_rows.h"

namespace ssm {
namespace {

// A workgroup takes 256 EACH consecutive pieces of the matrix, EACH a lane, all
// loaded before the first is written.  (32768 x 5120 bf16, us: packing 105,
// 113, 114, 119 with 1, 2, 4, 8 pieces; unpacking 88, 78, 80, 81.  Packing with
// nontemporal loads takes 89, but what unpacks after it 98.)
constexpr int kPackEach = 1, kUnpackEach = 2;

struct CkptP {
    uint8_t* x8;
    void* x;
    int64_t ld, pieces, scale_off;
    int P, W, W32;  // pieces of a row, columns, and columns with their padding
};

// Row and first value of the workgroup's piece i.
struct Place {
    int64_t row;
    int at;
};
__device__ __forceinline__ Place place(const CkptP& p, int64_t first_row, int first_piece, int i) {
    const uint32_t c = (uint32_t)(first_piece + i);
    return Place{first_row + c / (uint32_t)p.P, 8 * (int)(c % (uint32_t)p.P)};
}

template <typename T, Ends RAGGED>
__global__ __launch_bounds__(256) void ckpt8_pack(CkptP p) {
    constexpr int kEach = kPackEach, kPieces = 256 * kEach;
    const int64_t first = block_id() * kPieces, row0 = first / p.P;
    const int c0 = (int)(first - row0 * p.P);
    Piece<T> t[kEach];
    Place at[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int i = threadIdx.x + 256 * e;
        at[e] = place(p, row0, c0, i);
        t[e] = {};
        // pieces is a multiple of 4: a block's lanes go together
        if (first + i < p.pieces) load8<RAGGED>(t[e], static_cast<const T*>(p.x) + at[e].row * p.ld, at[e].at, p.W);
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        if (first + threadIdx.x + 256 * e >= p.pieces) return;
        float v[8];
        settle8<RAGGED>(t[e], at[e].at, p.W);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = t[e][j];
        CkptRow(p.x8, p.scale_off, p.W32, at[e].row, 0).store(at[e].at, v);
    }
}

template <typename T, Ends RAGGED>
__global__ __launch_bounds__(256) void ckpt8_unpack(CkptP p) {
    constexpr int kEach = kUnpackEach, kPieces = 256 * kEach;
    const int64_t first = block_id() * kPieces, row0 = first / p.P;
    const int c0 = (int)(first - row0 * p.P);
    CkptRow::Raw t[kEach];
    Place at[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int i = threadIdx.x + 256 * e;
        at[e] = place(p, row0, c0, i);
        if (first + i >= p.pieces) at[e].at = p.W;
        if (at[e].at < p.W) t[e] = CkptRow(p.x8, p.scale_off, p.W32, at[e].row, 0).load(at[e].at);
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        if (at[e].at >= p.W) continue;
        float v[8];
        t[e].values(v);
        store8<RAGGED>(static_cast<T*>(p.x) + at[e].row * p.ld, at[e].at, p.W, v);
    }
}

template <bool PACK>
int launch(uint8_t* x8, void* x, int64_t ld, int64_t M, int64_t W, int dtype, hipStream_t stream) {
    const int64_t W32 = ckpt8_width(W), pieces = M * (W32 / 8);
    if (!pieces) return SSM_OK;
    constexpr int64_t kPieces = 256 * (PACK ? kPackEach : kUnpackEach);
    const dim3 grid = block_grid((pieces + kPieces - 1) / kPieces);
    const CkptP p = {x8, x, ld, pieces, M * W32, (int)(W32 / 8), (int)W, (int)W32};
    auto go = [&](auto t) {
        using T = decltype(t);
        auto ends = [&](auto e) {
            if constexpr (PACK) ckpt8_pack<T, e.value><<<grid, 256, 0, stream>>>(p);
            else ckpt8_unpack<T, e.value><<<grid, 256, 0, stream>>>(p);
        };
        if (W < 8) ends(std::integral_constant<Ends, kTiny>());
        else if (W % 8) ends(std::integral_constant<Ends, kRagged>());
        else ends(std::integral_constant<Ends, kWhole>());
    };
    if (dtype == SSM_BF16) go(bf16_t());
    else go(float());
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // namespace

int launch_ckpt8_pack(const void* x, int64_t ld, int64_t M, int64_t W, int dtype, uint8_t* out,
                      hipStream_t stream) {
    return launch<true>(out, const_cast<void*>(x), ld, M, W, dtype, stream);
}

int launch_ckpt8_unpack(const uint8_t* x8, void* x, int64_t ld, int64_t M, int64_t W, int dtype,
                        hipStream_t stream) {
    return launch<false>(const_cast<uint8_t*>(x8), x, ld, M, W, dtype, stream);
}

}  // namespace ssm
