// Device helpers of the row kernels (norm_gated.hip, norm_residual.hip): a
// unit, one (row, group), is held in registers by L lanes of a wave (L = 8,
// 16, 32, 64) or, with L = 0, by a whole workgroup.  Lane t of n holds the
// 8-value pieces t, t + n, ... of the unit.  Pieces are loaded and stored
// whole at the element's own alignment (gfx950 takes 16-byte accesses at any),
// the last one value by value where the width is not a multiple of 8.
#pragma once

#include "ckpt8.h"

namespace ssm {

constexpr int kRowThreads = 256;  // workgroup of the kernels with L > 0

template <typename T>
struct Piece {
    T v[8];
    __device__ __forceinline__ float operator[](int j) const { return to_f32(v[j]); }
};

template <typename T>
__device__ __forceinline__ Piece<T> load8(const T* p, int n) {
    Piece<T> r;
    if (n >= 8) {
        __builtin_memcpy(&r, p, sizeof r);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.v[j] = j < n ? p[j] : T(0);
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void store8(T* p, int n, const float v[8]) {
    if (n >= 8) {
        Piece<T> r;
#pragma unroll
        for (int j = 0; j < 8; ++j) store_io(&r.v[j], v[j]);
        __builtin_memcpy(p, &r, sizeof r);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) store_io(p + j, v[j]);
    }
}

// the value as it is stored in T
__device__ __forceinline__ float as_stored(float v, float) { return v; }
__device__ __forceinline__ float as_stored(float v, bf16_t) { return to_f32(bf16_rne(v)); }

// Sum over the unit's lanes, in every one of them; a fixed order.  lds: 32
// floats for L = 0; turn alternates between calls, so that one barrier a call
// is enough (a wave is never more than one call ahead of another).
template <int L>
__device__ __forceinline__ float unit_sum(float v, float* lds, int turn) {
    constexpr int N = L == 0 ? 64 : L;
    v += quad_xor1(v);
    v += quad_xor2(v);
#pragma unroll
    for (int m = 4; m < N; m *= 2) v += __shfl_xor(v, m);
    if constexpr (L == 0) {
        const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6;
        if (waves > 1) {
            float* s = lds + 16 * (turn & 1);
            if ((threadIdx.x & 63) == 0) s[wave] = v;
            __syncthreads();
            v = 0.0f;
            for (int i = 0; i < waves; ++i) v += s[i];
        }
    }
    return v;
}

// Workgroup number of a grid from block_grid: a launch may hold at most 2^32
// lanes along an axis, which a long matrix passes.
__device__ __forceinline__ int64_t block_id() { return blockIdx.x + (int64_t)gridDim.x * blockIdx.y; }
inline dim3 block_grid(int64_t blocks) {
    const int64_t x = blocks < (1 << 20) ? blocks : 1 << 20;
    return dim3((unsigned)x, (unsigned)((blocks + x - 1) / x));
}

struct UnitLane {
    int unit, lane, lanes;  // unit within the workgroup, this lane of it, lanes a unit
};
template <int L>
__device__ __forceinline__ UnitLane unit_lane() {
    if constexpr (L == 0) return UnitLane{0, (int)threadIdx.x, (int)blockDim.x};
    else return UnitLane{(int)threadIdx.x / L, (int)threadIdx.x % L, L};
}
template <int L>
constexpr int units_per_block() { return L == 0 ? 1 : kRowThreads / L; }

// A row of an 8-bit checkpoint from column c0 (a multiple of 32) on.
struct CkptRow {
    uint8_t* codes;
    uint8_t* scales;
};
__device__ __forceinline__ CkptRow ckpt_row(uint8_t* base, int64_t scale_off, int W32, int64_t row, int c0) {
    return CkptRow{base + row * W32 + c0, base + scale_off + row * (W32 / 32) + c0 / 32};
}
// Writes piece c; the four lanes of the block's quad call it together.
__device__ __forceinline__ void ckpt_store(const CkptRow& r, int c, const float v[8]) {
    uint32_t b;
    const uint2 code = ckpt8_encode(v, &b);
    *reinterpret_cast<uint2*>(r.codes + 8 * (int64_t)c) = code;
    if ((c & 3) == 0) r.scales[c >> 2] = uint8_t(b);
}
__device__ __forceinline__ void ckpt_load(const CkptRow& r, int c, float v[8]) {
    const uint2 code = *reinterpret_cast<const uint2*>(r.codes + 8 * (int64_t)c);
    ckpt8_decode(code, ckpt8_scale(r.scales[c >> 2]), v);
}

// Adds the units' column sums of a workgroup and writes them to dst, the
// columns of the group (Wg of them).  sm: kRowThreads * 8 floats for L > 0.
template <int L, int NC>
__device__ __forceinline__ void store_column_sums(float* dst, int Wg, const float acc[NC][8], float* sm) {
    const UnitLane ul = unit_lane<L>();
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = ul.lane + k * ul.lanes, n = Wg - 8 * c;
        float t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = acc[k][j];
        if constexpr (L != 0) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) sm[8 * threadIdx.x + j] = t[j];
            __syncthreads();
            for (int u = 1; u < units_per_block<L>(); ++u)
#pragma unroll
                for (int j = 0; j < 8; ++j) t[j] += sm[8 * (u * L + ul.lane) + j];
        }
        if (ul.unit == 0 && n > 0) store8(dst + 8 * (int64_t)c, n, t);
    }
}

template <int L_, int NC_>
struct RowShape {
    static constexpr int L = L_, NC = NC_;
};

// Host: calls f(RowShape) for a group width: the smallest unit that holds it
// (8, 16, 32 or 64 lanes with one piece each, a wave with two, then a
// workgroup with 1, 2 or 4 pieces a lane), so that narrow rows share a wave
// and wide ones keep every lane busy.
template <typename F>
int for_row_shape(int Wg, F&& f) {
    const int pieces = (Wg + 7) / 8;
    if (pieces <= 8) return f(RowShape<8, 1>{});
    if (pieces <= 16) return f(RowShape<16, 1>{});
    if (pieces <= 32) return f(RowShape<32, 1>{});
    if (pieces <= 64) return f(RowShape<64, 1>{});
    if (pieces <= 128) return f(RowShape<64, 2>{});
    if (pieces <= 1024) return f(RowShape<0, 1>{});
    if (pieces <= 2048) return f(RowShape<0, 2>{});
    return f(RowShape<0, 4>{});
}
// threads of the workgroup for that shape
template <typename RS>
int row_threads(int Wg) {
    if (RS::L) return kRowThreads;
    const int pieces = (Wg + 7) / 8;
    return ((pieces + RS::NC - 1) / RS::NC + 63) / 64 * 64;
}

}  // namespace ssm
