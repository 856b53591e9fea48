// The 8-bit checkpoint format, shared by the kernels that write and read it.
//
// A [rows][width] tensor is kept as e4m3 codes in blocks of 32 along the row,
// each block with one power-of-two scale byte:
//   k      = the smallest integer >= -127 with amax <= 448 * 2^k   (amax over
//            the block's finite values; 448 is the largest e4m3 value)
//   code   = e4m3(x * 2^-k), round to nearest even; a value that is not
//            finite is kept as NaN and leaves its neighbours as they are
//   byte   = k + 127
// (in the last octave of f32, k = 120, a magnitude is at most 240: 256 * 2^120
// would read back as infinity)
// A scale rounded up, and not to the power of two at or below amax, keeps the
// block's largest value in range: no value is clamped and every one is within
// half a step (2^-4 of itself, or 2^-10 * 2^k near zero).  The scale being a
// power of two, x * 2^-k and code * 2^k are exact, and code * 2^k fits bf16.
// In memory: codes [rows][W32], W32 = width rounded up to 32, zeros past
// width, then the bytes [rows][W32 / 32].
//
// A lane quantises 8 consecutive values; four neighbouring lanes hold a block
// and find its amax by two quad permutes.
#pragma once

#include "device_common.h"

namespace ssm {

constexpr int kCkptBlock = 32;

__device__ __forceinline__ float fmax_quad(float v) {
    v = fmaxf(v, quad_xor1(v));
    return fmaxf(v, quad_xor2(v));
}

// Scale byte of a block with largest finite magnitude amax >= 0: with amax =
// f * 2^e, 1 <= f < 2, k = e - 8, plus 1 where f > 1.75 = 448 / 256.
__device__ __forceinline__ uint32_t ckpt8_scale_byte(float amax) {
    const uint32_t bits = __float_as_uint(amax);
    const int b = int(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return uint32_t(b > 0 ? b : 0);
}

// 2^(b - 127); b = 0 is the subnormal 2^-127
__device__ __forceinline__ float ckpt8_scale(uint32_t b) {
    return __uint_as_float(b ? b << 23 : 0x400000u);
}

// Codes of this lane's 8 values; the four lanes of a quad call it together.
// byte receives the block's scale byte.
__device__ __forceinline__ uint2 ckpt8_encode(const float v[8], uint32_t* byte) {
    float x[8], m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        x[j] = v[j];
        m = fmaxf(m, fabsf(v[j]));  // a quiet NaN drops out here and converts to NaN below
    }
    m = fmax_quad(m);
    // a block that holds an infinity or a signalling NaN: find amax again
    if (__builtin_amdgcn_ballot_w64(!(m < __builtin_inff()))) {
        m = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool finite = __builtin_isfinite(v[j]);
            x[j] = finite ? v[j] : __builtin_nanf("");
            m = fmaxf(m, finite ? fabsf(v[j]) : 0.0f);
        }
        m = fmax_quad(m);
    }
    const uint32_t b = ckpt8_scale_byte(m);
    if (__builtin_amdgcn_ballot_w64(b == 247u)) {
        const float top = b == 247u ? __uint_as_float((247u + 7u) << 23 | 0x700000u) : __builtin_inff();  // 240 * 2^120
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (fabsf(x[j]) > top) x[j] = copysignf(top, x[j]);
    }
    const float inv = __uint_as_float((254u - b) << 23);
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * inv, x[1] * inv, lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * inv, x[3] * inv, lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4] * inv, x[5] * inv, hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6] * inv, x[7] * inv, hi, true);
    *byte = b;
    return make_uint2(uint32_t(lo), uint32_t(hi));
}

__device__ __forceinline__ void ckpt8_decode(uint2 c, float scale, float v[8]) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(int(c.x), false);
    const auto b = __builtin_amdgcn_cvt_pk_f32_fp8(int(c.x), true);
    const auto d = __builtin_amdgcn_cvt_pk_f32_fp8(int(c.y), false);
    const auto e = __builtin_amdgcn_cvt_pk_f32_fp8(int(c.y), true);
    v[0] = a[0] * scale, v[1] = a[1] * scale, v[2] = b[0] * scale, v[3] = b[1] * scale;
    v[4] = d[0] * scale, v[5] = d[1] * scale, v[6] = e[0] * scale, v[7] = e[1] * scale;
}

}  // namespace ssm
