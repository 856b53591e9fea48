// Internal interface of the losses over a vocabulary (vocab_api.hip checks the
// arguments and runs a call; the launchers take them as checked).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "device_common.h"
#include "ssm.h"

namespace ssm {

// The products' tiles: 64 of the summed axis a step, waves of 64 columns (n)
// by 64 or 128 rows (m).
constexpr int kVocabStep = 64;
constexpr int kVocabTile = 256;  // what tensors in the workspace are padded to

// What the small kernels need of a call.  `rows` are the rows that count, in
// order: row c of them is row rows[c] of h.
struct VocabRows {
    int N, D, V, K, Np;  // K: entries a row (1 for a target); Np: N rounded up to the tile
    int terms;           // bf16 terms of a value: 1, or 3 for f32
    const int32_t* id;   // [N][K]
    const float* logit;  // [N][K], NULL for a target
    const float* top_lse;
    float top_scale;
    int32_t* count;      // rows that count
    int32_t* rows;       // [Np]
    int32_t* pos;        // [N]: place among rows, kRowOut or kRowBad
    int32_t* kid;        // [Np][K] ids of the rows that count, -1 for an absent entry
};
constexpr int32_t kRowOut = -1, kRowBad = -2;

int launch_vocab_rows(const VocabRows& r, uint32_t* err, hipStream_t stream);

// Rows of src (rows [r0, r0 + n) or, with `rows`, those of the list) as bf16
// terms: plain [terms][ld_rows][width rounded up to 64], or turned
// [terms][width][ld_rows], both zero behind the data up to the next 64.
struct VocabPack {
    const void* src;
    int64_t ld;
    int dtype, width, n;
    int64_t r0;
    const int32_t *rows, *count;
    uint16_t* out;
    int64_t ld_rows, plane;
};
int launch_vocab_pack(const VocabPack& p, hipStream_t stream);
int launch_vocab_turn(const VocabPack& p, hipStream_t stream);

// The backward's factors of a row that counts: g_v = coef exp2(s2_v - lse2) and,
// at entry k's id, q_k - p_k (entries with the same id hold the same sum).
struct VocabCoef {
    VocabRows r;
    const float *logq, *loss, *lse, *d_loss, *d_lse;
    float scale;
    float *lse2, *coef;  // [Np]
    float *at;           // [Np][K]: g at entry k's id
};
int launch_vocab_coef(const VocabCoef& c, hipStream_t stream);

struct VocabJoin {
    VocabRows r;
    const float2* part;  // [parts][Np]: max, sum of exp2
    int parts;
    float2* state;       // [Np] of the pieces before, or NULL
    bool first, last;
    const float* slog;   // [Np][K] logits at the ids, times log2 e
    float *loss, *lse, *logq;
};
int launch_vocab_join(const VocabJoin& j, hipStream_t stream);

// g at the entries' ids within the piece [v0, v0 + P).
struct VocabPatch {
    VocabRows r;
    const float* at;
    int v0, P;
    uint16_t *g, *gt;  // [terms][Np][P], [terms][P][Np]
};
int launch_vocab_patch(const VocabPatch& p, hipStream_t stream);

// d_h from the sum over parts of the rows that count [parts][Np][Dp].
struct VocabDh {
    VocabRows r;
    const float* acc;
    int parts, Dp, io;
    void* d_h;
    int64_t ld;
};
int launch_vocab_dh(const VocabDh& d, hipStream_t stream);

// out[n][m] = sum_k A[m][k] B[n][k] over planes of bf16 terms, k in steps of 64.
enum VocabMode { kLogitsFwd, kLogitsBwd, kGradH, kGradW };
struct VocabGemm {
    int mode, terms;
    const uint16_t *a, *b;
    int64_t a_plane, b_plane, lda, ldb;
    int m, n, k;           // rows of A and of B, and length of the sum
    const int32_t* count;  // device: bounds n (kGradW: k)
    int64_t Np;
    // kLogitsFwd, kLogitsBwd
    float scale2;          // scale * log2 e
    int v0, K;
    float2* part;
    const int32_t* kid;
    float* slog;
    const float *lse2, *coef;
    uint16_t *g, *gt;
    int P;
    // kGradH, kGradW: out row n (from row0), splits of k
    void* out;
    int64_t ld_out, split_stride;
    int splits, out_dtype;
    bool accumulate;
};
int vocab_parts(int m, int n);  // partials of a kLogitsFwd product, at most m / 64 + 4
int launch_vocab_gemm(const VocabGemm& g, hipStream_t stream);

// v as bf16 terms: exact in three, each what the ones before leave with the low
// half cut off (no rounding passes the largest value); an infinity or a NaN is
// all in the first.
__device__ __forceinline__ void bf16_terms(float v, uint16_t (&t)[3]) {
    const uint32_t bits = __float_as_uint(v);
    const bool finite = fabsf(v) < __builtin_inff();
    t[0] = v != v ? 0x7fc0 : bits >> 16;
    const float left = finite ? v - __uint_as_float(bits & 0xffff0000u) : 0.0f;
    t[1] = __float_as_uint(left) >> 16;
    t[2] = __float_as_uint(left - __uint_as_float(__float_as_uint(left) & 0xffff0000u)) >> 16;
}

}  // namespace ssm
