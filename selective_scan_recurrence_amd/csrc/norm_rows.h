// Device helpers of the row kernels (norm_gated.hip, norm_residual.hip,
// ckpt8.hip).  A unit, one (row, group), is held in registers by L lanes of a
// wave (L = 4, 8, 16, 32, 64) or, with L = 0, by a whole workgroup; where that
// would leave many lanes idle, a workgroup holds a row with all its groups
// (SEGMENTS) and adds each group's lanes through LDS.  Lane t of n
// holds the 8-value pieces t, t + n, ... of the unit, as 16-byte accesses at
// the element's own alignment, which gfx950 takes.  A width that is not a
// multiple of 8 (RAGGED) leaves a last piece of s = width % 8 values: it is
// loaded as the unit's last 8 values and shifted down in registers when it is
// used, so that no load is divided or waits behind a branch, and stored value
// by value.
#pragma once

#include "ckpt8.h"

namespace ssm {

// Whether a unit is whole pieces, ends in a part of one, or is less than one
// (its values are then loaded one by one: kept apart, because where the two ways
// of loading meet in one kernel every load is waited for at once).
enum Ends { kWhole, kRagged, kTiny };

constexpr int kRowThreads = 256;  // workgroup of the kernels with L > 0

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

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
        for (int j = 0; j < 4; ++j) {
            const f32x2 pair = {v[2 * j], v[2 * j + 1]};
            d[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(pair, bf16x2));
        }
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

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// Calls whose matrices together pass the 256 MB last-level cache, where their
// outputs would not stay for a reader, may store past the caches.
constexpr int64_t kStreamBytes = int64_t(256) << 20;

// Loads the piece at value `at` of a unit of n values; nothing past its end.  A
// ragged end is in place only after settle8, which waits for the load.
template <Ends RAGGED, typename T>
__device__ __forceinline__ void load8(Piece<T>& r, const T* unit, int at, int n) {
    if constexpr (RAGGED == kWhole) {
        if (at < n) __builtin_memcpy(&r, unit + at, sizeof r);
    } else if constexpr (RAGGED == kRagged) {
        if (at < n) __builtin_memcpy(&r, unit + min(at, n - 8), sizeof r);
    } else if (at == 0) {
        T v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < n ? unit[j] : T(0);
        __builtin_memcpy(&r, v, sizeof r);
    }
}
template <Ends RAGGED, typename T>
__device__ __forceinline__ void settle8(Piece<T>& r, int at, int n) {
    if constexpr (RAGGED == kRagged) {
        // only the wave that holds the end has anything to shift
        const bool end = at < n && at + 8 > n;
        if (__builtin_amdgcn_ballot_w64(end)) r.shift(8 - n % 8, end);
    }
}
// Both, for what is used at once.
template <Ends RAGGED, typename T>
__device__ __forceinline__ void fetch8(Piece<T>& r, const T* unit, int at, int n) {
    load8<RAGGED>(r, unit, at, n);
    settle8<RAGGED>(r, at, n);
}

// STREAM: past the caches
template <Ends RAGGED, bool STREAM = false, typename T>
__device__ __forceinline__ void store8(T* unit, int at, int n, const float v[8]) {
    Piece<T> r;
    r.set(v);
    if (RAGGED ? at + 8 <= n : at < n) {
        if constexpr (STREAM) {
            u32x4_any q[sizeof r / 16];
            __builtin_memcpy(q, &r, sizeof r);
#pragma unroll
            for (int i = 0; i < (int)sizeof r / 16; ++i)
                __builtin_nontemporal_store(q[i], reinterpret_cast<u32x4_any*>(unit + at) + i);
        } else {
            __builtin_memcpy(unit + at, &r, sizeof r);
        }
    }
    if (RAGGED && at < n && at + 8 > n) {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (at + j < n) store_io(unit + at + j, v[j]);
    }
}

// the values as they are stored in T
template <typename T>
__device__ __forceinline__ void as_stored(const float in[8], float out[8]) {
    Piece<T> r;
    r.set(in);
#pragma unroll
    for (int j = 0; j < 8; ++j) out[j] = r[j];
}

// 1 / sqrt(v) on the transcendental unit (1 ulp; v is at least 2^-126)
__device__ __forceinline__ float rsqrt1(float v) { return __builtin_amdgcn_rsqf(v); }

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
// sum over the 16 lanes of a DPP row (N = 16), each half (N = 8) or quad (N = 4)
// of it, in every lane
template <int N>
__device__ __forceinline__ float sum16(float v) {
    v += quad_xor1(v);
    v += quad_xor2(v);
    if (N >= 8) v += dpp<0x141>(v);     // row_half_mirror: the other quad of 8
    if (N == 16) v += dpp<0x140>(v);    // row_mirror: the other half
    return v;
}

// Sum over a wave's lanes, in every one of them.
__device__ __forceinline__ float sum_halves(float v) {  // of 16 lanes' sums: over 32 lanes
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}
__device__ __forceinline__ float sum_wave(float v) {
    v = sum_halves(sum16<16>(v));
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// LDS of unit_sum: two halves that alternate between calls, so that a call's
// barriers also keep the next call's writes from this one's reads (a wave is
// never more than one call ahead of another).
template <int L, int NC, bool SEGMENTS>
struct SumMemory {
    static constexpr int kHalf = L ? 1 : SEGMENTS ? 2 * NC * 1024 : 16;
    float m[2 * kHalf];
    __device__ __forceinline__ void init() {
        if constexpr (L == 0 && !SEGMENTS) {
            if (threadIdx.x < 2 * kHalf) m[threadIdx.x] = 0.0f;
            __syncthreads();
        }
    }
};

struct Groups {
    int count, pieces;  // groups of a row, 8-value pieces of one
};

// sum[k]: the sum of v over the unit's lanes and pieces, in every lane; with
// SEGMENTS the sum over piece k's group.  The order is fixed.
template <int L, int NC, bool SEGMENTS>
__device__ __forceinline__ void unit_sum(const float v[NC], float sum[NC], SumMemory<L, NC, SEGMENTS>& lds, int turn,
                                         const int (&group)[NC], Groups groups) {
    if constexpr (SEGMENTS) {
        // the pieces' values, then wave w adds the groups w, w + waves, ...
        float* s = lds.m + lds.kHalf * (turn & 1);
        float* total = s + NC * 1024;
        const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
#pragma unroll
        for (int k = 0; k < NC; ++k) s[threadIdx.x + k * blockDim.x] = v[k];
        __syncthreads();
        for (int g = threadIdx.x >> 6; g < groups.count; g += waves) {
            float a = 0.0f;
            for (int i = lane; i < groups.pieces; i += 64) a += s[g * groups.pieces + i];
            a = sum_wave(a);
            if (lane == 0) total[g] = a;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NC; ++k) sum[k] = total[group[k]];
        return;
    }
    float a = v[0];
#pragma unroll
    for (int k = 1; k < NC; ++k) a += v[k];
    if constexpr (L == 4 || L == 8 || L == 16) a = sum16<L ? L : 16>(a);
    else if constexpr (L == 32) a = sum_halves(sum16<16>(a));
    else a = sum_wave(a);
    if constexpr (L == 0) {
        float* s = lds.m + lds.kHalf * (turn & 1);
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = a;
        __syncthreads();
        a = sum16<16>(s[threadIdx.x & 15]);
    }
#pragma unroll
    for (int k = 0; k < NC; ++k) sum[k] = a;
}

// Whether a sum of unit_sum's call `turn` is infinite in this wave or, where a
// workgroup shares them, in any of it: the same answer in all of its waves.
template <int L, int NC, bool SEGMENTS>
__device__ __forceinline__ bool any_infinite(const float sum[NC], SumMemory<L, NC, SEGMENTS>& lds, int turn, Groups groups) {
    bool infinite = sum[0] == __builtin_inff();
    if constexpr (SEGMENTS) {
        const float* total = lds.m + lds.kHalf * (turn & 1) + NC * 1024;
        infinite = false;
        for (int g = threadIdx.x & 63; g < groups.count; g += 64) infinite |= total[g] == __builtin_inff();
    }
    return __builtin_amdgcn_ballot_w64(infinite) != 0;
}

// rstd[k] = 1 / sqrt(mean v^2 + eps) over the unit (with SEGMENTS, piece k's
// group), v(k, j) being this lane's values and ss[k] the sum of piece k's
// squares; all lanes call it together.  From 2^64 / sqrt(n) on the squares of
// finite values may add up to infinity: then they are added again of 2^-80 v,
// whose squares stay below 2^112 for up to 2^15 values, and beside which eps is
// nothing.  Only such rows take the second sum, and those that hold an
// infinity, which keep rstd = 0.  The branch is marked as rare, which keeps its
// registers from the others' (residual forward of 8192 x 12288 bf16: 292 us
// without it, 291 so, 327 unmarked; gated of 32768 x 5120: 176 and 173).
template <int L, int NC, bool SEGMENTS, typename V>
__device__ __forceinline__ void unit_rstd(const float ss[NC], V&& v, float rstd[NC], SumMemory<L, NC, SEGMENTS>& lds,
                                          int& turn, const int (&group)[NC], Groups groups, float inv_n, float eps) {
    float sum[NC];
    unit_sum(ss, sum, lds, turn, group, groups);
#pragma unroll
    for (int k = 0; k < NC; ++k) rstd[k] = rsqrt1(sum[k] * inv_n + eps);
    if (__builtin_expect(any_infinite(sum, lds, turn++, groups), 0)) {
        float again[NC], small[NC];
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            again[k] = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) again[k] += (v(k, j) * 0x1p-80f) * (v(k, j) * 0x1p-80f);
        }
        unit_sum(again, small, lds, turn++, group, groups);
#pragma unroll
        for (int k = 0; k < NC; ++k)
            if (sum[k] == __builtin_inff()) rstd[k] = rsqrt1(small[k] * inv_n) * 0x1p-80f;
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

// A row of a matrix, moved on by whole rows.
template <typename T>
struct RowPtr {
    T* p;
    int64_t ld;
    __device__ __forceinline__ RowPtr(const void* base, int64_t ld_, int64_t row, int c0)
        : p(const_cast<T*>(static_cast<const T*>(base)) + row * ld_ + c0), ld(ld_) {}
    __device__ __forceinline__ void skip(int64_t rows) { p += rows * ld; }
};

// A row of an 8-bit checkpoint, from column c0 (a multiple of 32) on.
struct CkptRow {
    uint8_t *codes, *scales;
    int W32;
    __device__ __forceinline__ CkptRow(const uint8_t* base, int64_t scale_off, int w32, int64_t row, int c0)
        : codes(const_cast<uint8_t*>(base) + row * w32 + c0),
          scales(const_cast<uint8_t*>(base) + scale_off + row * (w32 / 32) + c0 / 32), W32(w32) {}
    __device__ __forceinline__ void skip(int64_t rows) {
        codes += rows * W32;
        scales += rows * (W32 / 32);
    }
    // Writes the piece at value `at`; the block's quad calls it together.
    __device__ __forceinline__ void store(int at, const float v[8]) const {
        uint32_t b;
        const uint2 code = ckpt8_encode(v, &b);
        *reinterpret_cast<uint2*>(codes + at) = code;
        if ((at & 31) == 0) scales[at / 32] = uint8_t(b);
    }
    struct Raw {
        uint2 code;
        uint32_t byte;
        __device__ __forceinline__ void values(float v[8]) const { ckpt8_decode(code, ckpt8_scale(byte), v); }
    };
    __device__ __forceinline__ Raw load(int at) const {
        return Raw{*reinterpret_cast<const uint2*>(codes + at), scales[at / 32]};
    }
};

// A tensor's piece or its checkpoint's, as loaded.
template <typename T>
union PieceOr8 {
    Piece<T> t;
    CkptRow::Raw c;
    template <Ends RAGGED>
    __device__ __forceinline__ void values(bool kept, float v[8], int at, int n) {
        if (kept) return c.values(v);
        settle8<RAGGED>(t, at, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = t[j];
    }
};

// Adds the units' column sums of a workgroup and writes them to dst, n columns.
// sm: kRowThreads * 8 floats for L > 0.
template <int L, int NC, Ends RAGGED>
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

template <int L_, int NC_, Ends RAGGED_, bool SEGMENTS_ = false>
struct RowShape {
    static constexpr int L = L_, NC = NC_;
    static constexpr Ends RAGGED = RAGGED_;
    static constexpr bool SEGMENTS = SEGMENTS_;
};

// The kernels that ask for a shape: 65 to 128 pieces suit them differently.
enum RowUse { kGatedFwd, kGatedBwd, kResidual };

// Host: the smallest unit that holds a group of so many pieces (4, 8, 16, 32 or
// 64 lanes with one piece each, a wave with two, then a workgroup with 1, 2 or
// 4 pieces a lane), so that narrow rows share a wave and wide ones keep every
// lane busy.  Where a wave with two pieces would leave up to half its lanes idle:
//  - the residual norm gives up to 96 pieces to 32 lanes with three each (131072
//    x 640 bf16: forward 1.04 -> 0.95 times a copy's time, backward 1.13 -> 0.97;
//    the gated backward would hold 300 registers and go from 1.65 to 2.15);
//  - the gated backward, short of registers with two pieces, gives them to a
//    workgroup of two waves when there are many rows (131072 x 640 1.63 -> 1.19,
//    x 1024 1.18 -> 0.95, 32768 x 768 1.52 -> 1.22; 16384 x 768 would go from
//    1.28 to 1.45, the gated forward at 150000 x 523 from 1.16 to 1.43).
template <Ends RAGGED, RowUse USE, typename F>
int for_unit_shape(int pieces, bool many, F&& f) {
    if (pieces <= 4) return f(RowShape<4, 1, RAGGED>{});
    if (pieces <= 8) return f(RowShape<8, 1, RAGGED>{});
    if (pieces <= 16) return f(RowShape<16, 1, RAGGED>{});
    if (pieces <= 32) return f(RowShape<32, 1, RAGGED>{});
    if (pieces <= 64) return f(RowShape<64, 1, RAGGED>{});
    if constexpr (USE == kResidual)
        if (pieces <= 96) return f(RowShape<32, 3, RAGGED>{});
    if (USE != kGatedBwd || !many)
        if (pieces <= 128) return f(RowShape<64, 2, RAGGED>{});
    if (pieces <= 1024) return f(RowShape<0, 1, RAGGED>{});
    if (pieces <= 2048) return f(RowShape<0, 2, RAGGED>{});
    return f(RowShape<0, 4, RAGGED>{});
}
// threads of the workgroup for that shape
template <typename RS>
int row_threads(int pieces) {
    return RS::L ? kRowThreads : ((pieces + RS::NC - 1) / RS::NC + 63) / 64 * 64;
}
// Whether a workgroup takes whole rows of G groups: where the lanes of the
// units would be used 1/8 worse.
inline bool row_segments(int W, int G) {
    if (G == 1 || (W / G) % 8 || W / 8 > 1024) return false;
    const int pieces = W / G / 8, row = W / 8;
    int lanes = 0;
    for_unit_shape<kWhole, kGatedFwd>(pieces, false, [&](auto rs) {
        using RS = decltype(rs);
        return lanes = RS::L ? RS::L * RS::NC : row_threads<RS>(pieces) * RS::NC;
    });
    return (double)row / ((row + 63) / 64 * 64) > 1.125 * pieces / lanes;
}
// Calls f(RowShape, threads, groups that are units of their own) for a norm.
template <RowUse USE, typename F>
int for_row_shape(int64_t M, int W, int G, F&& f) {
    const int Wg = W / G;
    const bool many = M >= 32768;
    auto unit = [&](auto rs) { return f(rs, row_threads<decltype(rs)>((Wg + 7) / 8), G); };
    if constexpr (USE != kResidual)
        if (row_segments(W, G)) {
            using RS = RowShape<0, 1, kWhole, true>;
            return f(RS{}, row_threads<RS>(W / 8), 1);
        }
    if (Wg < 8) return unit(RowShape<4, 1, kTiny>{});
    return Wg % 8 ? for_unit_shape<kRagged, USE>((Wg + 7) / 8, many, unit)
                  : for_unit_shape<kWhole, USE>(Wg / 8, many, unit);
}

// Slices of a forward, whose workgroups (slice, group) walk the rows: 16 waves
// on each of 256 compute units, fewer for fewer rows; 24 with SEGMENTS, whose
// workgroups wait twice a row.  (32768 x 5120 bf16, gated: 177, 176, 184, 222
// us with 12, 16, 24, 32 waves, one workgroup a row 420 us; 16384 x 5120 in 8
// groups with two checkpoints: 152, 138, 149 us with 16, 24, 32.)
template <typename RS>
int row_slices(int64_t M, int units, int threads) {
    const int64_t need = (M + units_per_block<RS::L>() - 1) / units_per_block<RS::L>();
    const int each = (RS::SEGMENTS ? 24 : 16) * 64 / threads;
    const int64_t most = 256 * (int64_t)(each > 0 ? each : 1) / units;
    return (int)(need < most ? need : most > 0 ? most : 1);
}

// The unit of a lane and, with SEGMENTS, the groups of its pieces.
template <typename RS>
struct RowLane {
    UnitLane ul;
    int c0, n;            // first column and columns of the unit
    int group[RS::NC];    // group of each piece
    __device__ __forceinline__ RowLane(int G, int Wg) : ul(unit_lane<RS::L>()) {
        c0 = RS::SEGMENTS ? 0 : (int)(blockIdx.x % G) * Wg;
        n = RS::SEGMENTS ? G * Wg : Wg;
#pragma unroll
        for (int k = 0; k < RS::NC; ++k)
            group[k] = !RS::SEGMENTS ? (int)(blockIdx.x % G) : ul.at(k) < n ? ul.at(k) / Wg : 0;
    }
    __device__ __forceinline__ int slice(int G) const { return RS::SEGMENTS ? blockIdx.x : blockIdx.x / G; }
    __device__ __forceinline__ int at(int k) const { return ul.at(k); }
};

// Calls step(present row, next row's place) for the rows of a unit below M,
// the workgroup's first rows being first, first + stride, ...: every unit
// makes the same number of turns (the last may have no row left).  The present
// row is a copy: two rows that swap their parts save its few moves but cost
// registers (backward of 16384 x 2560: 107 -> 124 us).
template <typename Row, typename F>
__device__ __forceinline__ void walk_rows(Row& next, int64_t first, int64_t M, int64_t stride, F&& step) {
    for (; first < M; first += stride) {
        Row present = next;
        step(present, next);
    }
}

}  // namespace ssm
