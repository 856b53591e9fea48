// Device helpers of the row kernels (norm_gated.hip, norm_residual.hip,
// ckpt8.hip).  A unit, one (row, group), is held in registers by L lanes of a
// wave (L = 8, 16, 32, 64) or, with L = 0, by a whole workgroup.  Lane t of n
// holds the 8-value pieces t, t + n, ... of the unit, as 16-byte accesses at
// the element's own alignment, which gfx950 takes.  A width that is not a
// multiple of 8 (RAGGED) leaves a last piece of s = width % 8 values: it is
// loaded as the unit's last 8 values and shifted down in registers, so that
// no load is divided or waits behind a branch, and stored value by value.
#pragma once

#include "ckpt8.h"

namespace ssm {

constexpr int kRowThreads = 256;  // workgroup of the kernels with L > 0

template <typename T>
struct Piece;
template <>
struct Piece<bf16_t> {
    uint32_t d[4];
    __device__ __forceinline__ float operator[](int j) const {
        return __uint_as_float(j & 1 ? d[j / 2] & 0xffff0000u : d[j / 2] << 16);
    }
    // drops the first n values (n < 8) where on, zeros behind them
    __device__ __forceinline__ void shift(int n, bool on) {
        const uint32_t z = 0;
        if (n & 4) {
            d[0] = on ? d[2] : d[0], d[1] = on ? d[3] : d[1];
            d[2] = on ? z : d[2], d[3] = on ? z : d[3];
        }
        if (n & 2) {
#pragma unroll
            for (int j = 0; j < 4; ++j) d[j] = on ? (j < 3 ? d[j + 1] : z) : d[j];
        }
        if (n & 1) {
#pragma unroll
            for (int j = 0; j < 4; ++j) d[j] = on ? (j < 3 ? d[j] >> 16 | d[j + 1] << 16 : d[j] >> 16) : d[j];
        }
    }
    __device__ __forceinline__ void set(const float v[8]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = uint32_t(bf16_rne(v[2 * j])) | uint32_t(bf16_rne(v[2 * j + 1])) << 16;
    }
};
template <>
struct Piece<float> {
    float d[8];
    __device__ __forceinline__ float operator[](int j) const { return d[j]; }
    __device__ __forceinline__ void shift(int n, bool on) {
#pragma unroll
        for (int s = 4; s > 0; s /= 2)
            if (n & s) {
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] = on ? (j + s < 8 ? d[j + s] : 0.0f) : d[j];
            }
    }
    __device__ __forceinline__ void set(const float v[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = v[j];
    }
};

// Loads the piece at value `at` of a unit of n values; nothing past its end.
template <bool RAGGED, typename T>
__device__ __forceinline__ void load8(Piece<T>& r, const T* unit, int at, int n) {
    if constexpr (!RAGGED) {
        if (at < n) __builtin_memcpy(&r, unit + at, sizeof r);
    } else if (n >= 8) {
        if (at < n) __builtin_memcpy(&r, unit + min(at, n - 8), sizeof r);
        r.shift(8 - n % 8, at < n && at + 8 > n);
    } else if (at == 0) {
        T v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < n ? unit[j] : T(0);
        __builtin_memcpy(&r, v, sizeof r);
    }
}

template <bool RAGGED, typename T>
__device__ __forceinline__ void store8(T* unit, int at, int n, const float v[8]) {
    Piece<T> r;
    r.set(v);
    if (RAGGED ? at + 8 <= n : at < n) __builtin_memcpy(unit + at, &r, sizeof r);
    if (RAGGED && at < n && at + 8 > n) {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (at + j < n) store_io(unit + at + j, v[j]);
    }
}

// the value as it is stored in T
__device__ __forceinline__ float as_stored(float v, float) { return v; }
__device__ __forceinline__ float as_stored(float v, bf16_t) { return to_f32(bf16_rne(v)); }

// 1 / sqrt(v) on the transcendental unit (1 ulp; v is at least 2^-126)
__device__ __forceinline__ float rsqrt1(float v) { return __builtin_amdgcn_rsqf(v); }

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
// sum over the 16 lanes of a DPP row (N = 16) or each half of it (N = 8), in every lane
template <int N>
__device__ __forceinline__ float sum16(float v) {
    v += quad_xor1(v);
    v += quad_xor2(v);
    v += dpp<0x141>(v);                 // row_half_mirror: the other quad of 8
    if (N == 16) v += dpp<0x140>(v);    // row_mirror: the other half
    return v;
}

// Sum over the unit's lanes, in every one of them; a fixed order.  lds: 32
// floats for L = 0, zero at first; turn alternates between calls, so that one
// barrier a call is enough (a wave is never more than one call ahead of
// another).
template <int L>
__device__ __forceinline__ float unit_sum(float v, float* lds, int turn) {
    v = sum16<L == 8 ? 8 : 16>(v);
    if constexpr (L == 0 || L >= 32) {
        const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
    if constexpr (L == 0 || L == 64) {
        const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
    if constexpr (L == 0) {
        float* s = lds + 16 * (turn & 1);
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
        __syncthreads();
        v = sum16<16>(s[threadIdx.x & 15]);
    }
    return v;
}
// Clears unit_sum's memory.
template <int L>
__device__ __forceinline__ void unit_sum_init(float* lds) {
    if constexpr (L == 0) {
        if (threadIdx.x < 32) lds[threadIdx.x] = 0.0f;
        __syncthreads();
    }
}

// A launch may hold at most 2^32 lanes along an axis, which a long matrix
// passes: a grid in x and y, and the workgroup's number in it.
__device__ __forceinline__ int64_t block_id() { return blockIdx.x + (int64_t)gridDim.x * blockIdx.y; }
inline dim3 block_grid(int64_t blocks) {
    const int64_t x = blocks < (1 << 20) ? blocks : 1 << 20;
    return dim3((unsigned)x, (unsigned)((blocks + x - 1) / x));
}

struct UnitLane {
    int unit, lane, lanes;  // unit within the workgroup, this lane of it, lanes a unit
    __device__ __forceinline__ int at(int k) const { return 8 * (lane + k * lanes); }  // value of piece k
};
template <int L>
__device__ __forceinline__ UnitLane unit_lane() {
    if constexpr (L == 0) return UnitLane{0, (int)threadIdx.x, (int)blockDim.x};
    else return UnitLane{(int)threadIdx.x / L, (int)threadIdx.x % L, L};
}
template <int L>
constexpr int units_per_block() { return L == 0 ? 1 : kRowThreads / L; }

// An 8-bit checkpoint, from column c0 (a multiple of 32) on.
struct Ckpt {
    uint8_t *codes, *scales;
    int W32;
    __device__ __forceinline__ Ckpt(uint8_t* base, int64_t scale_off, int w32, int c0)
        : codes(base + c0), scales(base + scale_off + c0 / 32), W32(w32) {}
    // Writes the piece at value `at` of a row; the block's quad calls it together.
    __device__ __forceinline__ void store(int64_t row, int at, const float v[8]) const {
        uint32_t b;
        const uint2 code = ckpt8_encode(v, &b);
        *reinterpret_cast<uint2*>(codes + row * W32 + at) = code;
        if ((at & 31) == 0) scales[row * (W32 / 32) + at / 32] = uint8_t(b);
    }
    struct Raw {
        uint2 code;
        uint32_t byte;
        __device__ __forceinline__ void values(float v[8]) const { ckpt8_decode(code, ckpt8_scale(byte), v); }
    };
    __device__ __forceinline__ Raw load(int64_t row, int at) const {
        return Raw{*reinterpret_cast<const uint2*>(codes + row * W32 + at), scales[row * (W32 / 32) + at / 32]};
    }
};

// A tensor's piece or its checkpoint's, as loaded.
template <typename T>
union PieceOr8 {
    Piece<T> t;
    Ckpt::Raw c;
};

// Adds the units' column sums of a workgroup and writes them to dst, n columns.
// sm: kRowThreads * 8 floats for L > 0.
template <int L, int NC, bool RAGGED>
__device__ __forceinline__ void store_column_sums(float* dst, int n, const float acc[NC][8], float* sm) {
    const UnitLane ul = unit_lane<L>();
#pragma unroll
    for (int k = 0; k < NC; ++k) {
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
        if (ul.unit == 0) store8<RAGGED>(dst, ul.at(k), n, t);
    }
}

template <int L_, int NC_, bool RAGGED_>
struct RowShape {
    static constexpr int L = L_, NC = NC_;
    static constexpr bool RAGGED = RAGGED_;
};

// Host: calls f(RowShape) for a group width: the smallest unit that holds it
// (8, 16, 32 or 64 lanes with one piece each, a wave with two, then a
// workgroup with 1, 2 or 4 pieces a lane), so that narrow rows share a wave
// and wide ones keep every lane busy.
template <bool RAGGED, typename F>
int for_row_shape_of(int pieces, F&& f) {
    if (pieces <= 8) return f(RowShape<8, 1, RAGGED>{});
    if (pieces <= 16) return f(RowShape<16, 1, RAGGED>{});
    if (pieces <= 32) return f(RowShape<32, 1, RAGGED>{});
    if (pieces <= 64) return f(RowShape<64, 1, RAGGED>{});
    if (pieces <= 128) return f(RowShape<64, 2, RAGGED>{});
    if (pieces <= 1024) return f(RowShape<0, 1, RAGGED>{});
    if (pieces <= 2048) return f(RowShape<0, 2, RAGGED>{});
    return f(RowShape<0, 4, RAGGED>{});
}
template <typename F>
int for_row_shape(int Wg, F&& f) {
    return Wg % 8 ? for_row_shape_of<true>((Wg + 7) / 8, f) : for_row_shape_of<false>(Wg / 8, f);
}
// threads of the workgroup for that shape
template <typename RS>
int row_threads(int Wg) {
    if (RS::L) return kRowThreads;
    const int pieces = (Wg + 7) / 8;
    return ((pieces + RS::NC - 1) / RS::NC + 63) / 64 * 64;
}

// Slices of a kernel whose workgroups (slice, group) walk the rows: 16 waves on
// each of 256 compute units, fewer for fewer rows.  (32768 x 5120 bf16, gated:
// 177, 176, 184, 222 us with 12, 16, 24, 32 waves; one workgroup a row 420 us.)
constexpr int kRowWaves = 16;
template <typename RS>
int row_slices(int64_t M, int G, int threads) {
    const int64_t need = (M + units_per_block<RS::L>() - 1) / units_per_block<RS::L>();
    const int64_t most = 256 * (int64_t)(kRowWaves * 64 / threads > 0 ? kRowWaves * 64 / threads : 1) / G;
    return (int)(need < most ? need : most > 0 ? most : 1);
}

}  // namespace ssm
