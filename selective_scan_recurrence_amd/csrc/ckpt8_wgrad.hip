// Weight gradient of a projection whose input was kept as an 8-bit checkpoint:
//   dw[o][c] = sum_m dy[m][o] x[m][c] (+ dw[o][c]),  x = code * 2^k.
// Both operands run along the summed axis m with their slow axis, so both
// have to be transposed for the MFMA, whose lanes want 8 consecutive m of one
// column.  A code times its scale fits bf16, so the products are exact; an f32
// dy enters as three bf16 terms (24 bits), with three MFMAs.
//
// A workgroup (4 waves) owns 256 (o) x 128 (c) of dw, wave w the rows 64w ..
// 64w + 63, and walks m in steps of 64:
//   dy: a wave's 64 columns are its own, so they go from memory to its
//     registers past LDS: lane 16g + i loads columns 4i .. 4i + 3 of the rows
//     8g .. 8g + 7 of a 32-row half step and pairs rows with one byte permute
//     a register.  Its four columns belong to four MFMA tiles: tile t takes
//     columns 4i + t, i = 0 .. 15.
//   x: all four waves need all 128 columns: a thread converts 8 rows of 4
//     columns, pairs them the same way and writes a column's 8 rows as one
//     16-byte piece to LDS, which the waves read as MFMA operands.  Column c's
//     piece q sits at c' * 128 + 16 (q ^ (c / 4 % 8)) bytes, c' = c ^ (c / 32
//     % 2): the 8 lanes of a write (c = 4 l + t) and of a read (tile j, lane
//     i: c = 4i + j % 4 + 64 (j / 4)) then meet 8 different 16-byte columns.
// With few tiles the rows are split over workgroups, each of which leaves an
// f32 partial in the workspace, and a second kernel adds them in order.
//
// Bound by the matrix units, two workgroups a CU: 8192 rows, 4096 x 4096, bf16
// dy, where 512 tiles fill the CUs at once, 242 us = 1136 TFLOP/s over one set of
// tensors, which the last-level cache holds, and 273 us = 1007 over three in turn
// (a library product of 8192^3 in bf16 reaches 1251); 8192 rows, 10576 x 2560,
// 497 and 514 us = 892 and 863 TFLOP/s (840 tiles: a round of 512 and a part of
// one; a library product of the same sizes with x in bf16 takes 565 to 578 us).  Leaving out half of the dy loads
// there gains 10% (its rows start off the cache lines), the loads of scales or
// the conversions nothing; narrower tiles that fill the rounds better lose
// (columns 112: 544 - 579 us, 96: 670), and so do other orders of the loads and
// the MFMAs.  f32 dy, 4096 rows, 5120 x 2560: 450 us = 716 TFLOP/s of its three
// MFMAs a product: 400 tiles on 256 places, one workgroup a CU with 400 registers
// a lane, whose one wave a SIMD splits dy and multiplies in turn.
#include <type_traits>

#include "block_internal.h"
#include "norm_rows.h"
#include "row_split.h"

namespace ssm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

struct WgradP {
    const void* dy;
    const uint8_t* x8;
    float* out;        // dw, or the partials [splits][O][W]
    int64_t ld, scale_off;
    int M, W, W32, O;
    int tiles_c, tiles;   // tiles along c, tiles in all
    int rows;             // rows a split, a multiple of kTM
    bool accumulate;
};

// dword with row a's 16-bit half h below row b's
__device__ __forceinline__ uint32_t pair_rows(uint32_t a, uint32_t b, int h) {
    return __builtin_amdgcn_perm(b, a, h ? 0x07060302u : 0x05040100u);
}

// A descriptor without a bound: whole steps only load what is there.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* base) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, 0x7fffffff, 0x00020000);
}

// A half step's dy of a lane: rows 8g .. 8g + 7, 4 columns.
template <typename T>
struct DyRaw;
template <>
struct DyRaw<bf16_t> {
    static constexpr int kTerms = 1;
    u32x2 r[8];
    __device__ __forceinline__ void load(int j, __amdgpu_buffer_rsrc_t b, int at, int row) {
        r[j] = __builtin_amdgcn_raw_buffer_load_b64(b, at, row, 0);
    }
    __device__ __forceinline__ void zero(int j) { r[j] = u32x2{0, 0}; }
    __device__ __forceinline__ void frags(u32x4 (&f)[1][4]) const {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int p = 0; p < 4; ++p) f[0][t][p] = pair_rows(r[2 * p][t / 2], r[2 * p + 1][t / 2], t & 1);
    }
};
template <>
struct DyRaw<float> {
    static constexpr int kTerms = 3;
    u32x4 r[8];
    __device__ __forceinline__ void load(int j, __amdgpu_buffer_rsrc_t b, int at, int row) {
        r[j] = __builtin_amdgcn_raw_buffer_load_b128(b, at, row, 0);
    }
    __device__ __forceinline__ void zero(int j) { r[j] = u32x4{0, 0, 0, 0}; }
    // v = hi + mid + lo, the three bytes of its significand: each what is left
    // with the low half cut off, so exact, and no rounding passes the largest
    // value.  An infinity or a NaN is all in hi.
    __device__ __forceinline__ void frags(u32x4 (&f)[3][4]) const {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                uint32_t w[3][2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float v = __uint_as_float(r[2 * p + h][t]);
                    const bool finite = fabsf(v) < __builtin_inff();
                    const uint32_t top = r[2 * p + h][t] & 0xffff0000u;
                    w[0][h] = v != v ? 0x7fc00000u : top;
                    const float left = finite ? v - __uint_as_float(top) : 0.0f;
                    w[1][h] = __float_as_uint(left) & 0xffff0000u;
                    w[2][h] = __float_as_uint(left - __uint_as_float(w[1][h]));
                }
#pragma unroll
                for (int n = 0; n < 3; ++n) f[n][t][p] = pair_rows(w[n][0], w[n][1], 1);
            }
    }
};

// NARROW: fewer than 4 columns of dy in all, loaded one by one.
template <typename T, bool NARROW>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void wgrad_tile(WgradP p) {
    constexpr int NT = DyRaw<T>::kTerms;
    __shared__ __attribute__((aligned(16))) uint8_t lds[2][kTC * kTM * 2];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i16 = lane & 15, g = lane >> 4;
    // XCD-ordered numbering (workgroups are dealt to the 8 XCDs in turn): an
    // XCD's workgroups are neighbouring tiles, c fastest, that share dy and x
    const uint32_t n_wg = gridDim.x, pid = blockIdx.x;
    const uint32_t per = n_wg / 8, extra = n_wg % 8, xcd = pid % 8;
    const uint32_t id = xcd * per + min(xcd, extra) + pid / 8;
    const int split = id / p.tiles, tile = id % p.tiles;
    const int o0 = tile / p.tiles_c * kTO + 64 * wave, c0 = tile % p.tiles_c * kTC;
    const int m_begin = split * p.rows, m_end = part_end(p.M, p.rows, split);

    // dy: columns past O are never stored, so a lane past the end takes the
    // last four.  A step's rows past the end (LAST) are loaded from the last
    // row and zeroed, so that nothing of them reaches a sum.  Whole steps load
    // from a scalar base that moves with the step, a scalar row offset and a
    // lane offset that stays.
    const int col = NARROW ? 0 : min(o0 + 4 * i16, p.O - 4);
    const T* dy = static_cast<const T*>(p.dy);
    const int dy_row = (int)p.ld * (int)sizeof(T), dy_at = 8 * g * dy_row + col * (int)sizeof(T);
    auto load_dy = [&](DyRaw<T>& d, int m0, int ks, auto rsrc, auto last) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (NARROW) {
                T v[4];
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    v[t] = dy[(int64_t)min(m0 + 32 * ks + 8 * g + j, p.M - 1) * p.ld + min(t, p.O - 1)];
                __builtin_memcpy(&d.r[j], v, sizeof v);
            } else if constexpr (last.value) {
                __builtin_memcpy(&d.r[j], dy + (int64_t)min(m0 + 32 * ks + 8 * g + j, m_end - 1) * p.ld + col,
                                 sizeof d.r[j]);
            } else {
                d.load(j, rsrc, dy_at, (32 * ks + j) * dy_row);
            }
            if (last.value && m0 + 32 * ks + 8 * g + j >= m_end) d.zero(j);
        }
    };
    // x: thread (octet of rows, 4 columns); columns past W32 are never stored
    const int cl = tid & 31, octet = tid >> 5;
    const int xc = min(c0 + 4 * cl, p.W32 - 4), blocks = p.W32 / 32;
    const int x_at = 8 * octet * p.W32 + xc, s_at = 8 * octet * blocks + xc / 32;
    uint32_t xr[8], xs[8];
    auto load_x = [&](int m0, auto codes, auto scales, auto last) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (last.value) {
                const int m = m0 + 8 * octet + j, r = min(m, m_end - 1);
                __builtin_memcpy(&xr[j], p.x8 + (int64_t)r * p.W32 + xc, 4);
                xs[j] = p.x8[p.scale_off + (int64_t)r * blocks + xc / 32];
                if (m >= m_end) xr[j] = 0;
            } else {
                xr[j] = __builtin_amdgcn_raw_buffer_load_b32(codes, x_at, j * p.W32, 0);
                xs[j] = __builtin_amdgcn_raw_buffer_load_b8(scales, s_at, j * blocks, 0);
            }
        }
    };
    auto store_x = [&](uint8_t* buf) {
        uint32_t v[8][2];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = __uint_as_float(xs[j] << 23);
            v[j][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)xr[j], s, false));
            v[j][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)xr[j], s, true));
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            u32x4 w;
#pragma unroll
            for (int q = 0; q < 4; ++q) w[q] = pair_rows(v[2 * q][t / 2], v[2 * q + 1][t / 2], t & 1);
            const int c = 4 * cl + t;
            *reinterpret_cast<u32x4*>(buf + (c ^ (c >> 5 & 1)) * 128 + 16 * (octet ^ (cl & 7))) = w;
        }
    };

    DyRaw<T> raw[2];
    f32x4 acc[4][8];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[t][j] = f32x4{0, 0, 0, 0};

    // one half step: rows 32 ks .. 32 ks + 31 of the buffer
    auto multiply = [&](const u32x4 (&a)[NT][4], const uint8_t* buf, int ks) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = 4 * i16 + (j & 3) + 64 * (j >> 2);
            const u32x4 b = *reinterpret_cast<const u32x4*>(
                buf + (c ^ (c >> 5 & 1)) * 128 + 16 * ((g + 4 * ks) ^ (i16 & 7)));
#pragma unroll
            for (int n = NT - 1; n >= 0; --n)
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    acc[t][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, a[n][t]), __builtin_bit_cast(bf16x8, b), acc[t][j], 0, 0, 0);
        }
    };

    // Buffers alternate: step n + 1 is loaded while step n is multiplied, and
    // written to the other buffer after it, with one barrier a step.  A half
    // step's dy is turned into operands first, so that its registers take the
    // next one's.  In f32 the loads are pinned there, a whole step ahead of their
    // use (467 against 507 us for 4096 rows, 2560 x 5120); in bf16, where two
    // waves share a SIMD, the scheduler does better by itself (235 against 262 us
    // for 8192 rows, 5120 x 2560).
    auto step = [&](int next, int cur, auto last) {  // multiplies buffer cur, loads the step at next
        u32x4 a[NT][4];
        const auto rows = rsrc_of(dy + (int64_t)next * p.ld);
        load_x(next, rsrc_of(p.x8 + (int64_t)next * p.W32), rsrc_of(p.x8 + p.scale_off + (int64_t)next * blocks), last);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            raw[ks].frags(a);
            load_dy(raw[ks], next, ks, rows, last);
            if constexpr (NT > 1) __builtin_amdgcn_sched_barrier(0);
            multiply(a, lds[cur], ks);
            if constexpr (NT > 1) __builtin_amdgcn_sched_barrier(0);
        }
        store_x(lds[cur ^ 1]);
        __syncthreads();
    };
    constexpr std::false_type whole{};
    constexpr std::true_type partial{};
    auto load = [&](int m0, auto last) {
        const auto rows = rsrc_of(dy + (int64_t)m0 * p.ld);
        load_x(m0, rsrc_of(p.x8 + (int64_t)m0 * p.W32), rsrc_of(p.x8 + p.scale_off + (int64_t)m0 * blocks), last);
        load_dy(raw[0], m0, 0, rows, last);
        load_dy(raw[1], m0, 1, rows, last);
    };
    if (m_begin < m_end) {
        int m = m_begin, cur = 0;
        if (m + kTM <= m_end) load(m, whole);
        else load(m, partial);
        store_x(lds[0]);
        __syncthreads();
        for (; m + 2 * kTM <= m_end; m += kTM, cur ^= 1) step(m + kTM, cur, whole);
        if (m + kTM < m_end) {
            step(m + kTM, cur, partial);
            cur ^= 1;
        }
        u32x4 a[NT][4];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            raw[ks].frags(a);
            multiply(a, lds[cur], ks);
        }
    }

    // lane 16g + i holds rows 16g + 4r + t (r = 0 .. 3) and, over j % 4, four
    // neighbouring columns
    float* out = p.out + (int64_t)split * p.O * p.W;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int want = o0 + 16 * g + 4 * r;  // the columns of dy that lane 4g + r stands for
            const int o = (NARROW ? want : min(want, p.O - 4)) + t;
            if (o < want || o >= p.O) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = c0 + 64 * h + 4 * i16, n = p.W - c;
                if (n <= 0) continue;
                float v[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = acc[t][4 * h + q][r];
                float* at = out + (int64_t)o * p.W + c;
                if (n >= 4) {
                    float4 s = make_float4(v[0], v[1], v[2], v[3]);
                    if (p.accumulate) {
                        float4 u;
                        __builtin_memcpy(&u, at, 16);
                        s = make_float4(s.x + u.x, s.y + u.y, s.z + u.z, s.w + u.w);
                    }
                    __builtin_memcpy(at, &s, 16);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (q < n) at[q] = p.accumulate ? at[q] + v[q] : v[q];
                }
            }
        }
}

// dw[e] = sum_s part[s][e] (+ dw[e]): SL lanes share an element, lane l taking
// the parts l, l + SL, ..., and are added in order.
template <int SL>
__global__ __launch_bounds__(256) void wgrad_join(const float* __restrict__ part, float* dw, int64_t n, int S,
                                                  bool accumulate) {
    constexpr int E = 256 / SL;
    __shared__ float sm[SL > 1 ? SL : 1][E];
    const int l = threadIdx.x / E, i = threadIdx.x % E;
    const int64_t e = (int64_t)blockIdx.x * E + i;
    float v = 0.0f;
    if (e < n)
#pragma unroll 4
        for (int s = l; s < S; s += SL) v += part[s * n + e];
    if constexpr (SL > 1) {
        sm[l][i] = v;
        __syncthreads();
        if (l > 0) return;
#pragma unroll
        for (int s = 1; s < SL; ++s) v += sm[s][i];
    }
    if (e < n) dw[e] = accumulate ? dw[e] + v : v;
}

}  // namespace

size_t ckpt8_wgrad_workspace_bytes(int64_t M, int64_t W, int64_t O, int dtype) {
    const RowSplit s = split_rows(M, W, O, dtype);
    return s.count > 1 ? (size_t)s.count * W * O * 4 : 0;
}

int launch_ckpt8_wgrad(const void* dy, int64_t ld, const uint8_t* x8, float* dw, int64_t M, int64_t W,
                       int64_t O, int dtype, bool accumulate, void* ws, hipStream_t stream) {
    const RowSplit s = split_rows(M, W, O, dtype);
    const int64_t W32 = ckpt8_width(W);
    const int tiles_c = (int)((W + kTC - 1) / kTC);
    const int64_t tiles = tiles_c * ((O + kTO - 1) / kTO);
    const bool joined = s.count > 1;
    WgradP p = {dy, x8, joined ? static_cast<float*>(ws) : dw, ld, M * W32, (int)M, (int)W, (int)W32, (int)O,
                tiles_c, (int)tiles, s.rows, !joined && accumulate};
    const unsigned grid = (unsigned)(tiles * s.count);
    if (dtype == SSM_BF16) {
        if (O < 4) wgrad_tile<bf16_t, true><<<grid, 256, 0, stream>>>(p);
        else wgrad_tile<bf16_t, false><<<grid, 256, 0, stream>>>(p);
    } else {
        if (O < 4) wgrad_tile<float, true><<<grid, 256, 0, stream>>>(p);
        else wgrad_tile<float, false><<<grid, 256, 0, stream>>>(p);
    }
    if (joined) {
        const int64_t n = W * O;
        const float* part = static_cast<float*>(ws);
        if (s.count <= 8) wgrad_join<1><<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(part, dw, n, s.count, accumulate);
        else wgrad_join<8><<<(unsigned)((n + 31) / 32), 256, 0, stream>>>(part, dw, n, s.count, accumulate);
    }
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // namespace ssm
