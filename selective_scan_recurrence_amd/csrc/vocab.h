// Internal interface of the losses over a vocabulary (vocab_api.hip checks the
// arguments and runs a call; the launchers take them as checked).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "device_common.h"
#include "ssm.h"
#include "vocab_plan.h"

namespace ssm {

constexpr int kVocabStep = 64;    // of the summed axis, a step of the products' tiles
constexpr int kVocabTile = 256;   // what tensors in the workspace are padded to

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
    int32_t* pos;        // [N]: place among rows, kRowOut or kRowBad (NULL: not listed, rows keep their places)
    int32_t* kid;        // [K][Np] ids of the rows that count, -1 for an absent entry
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

// The backward's factors of a row that counts: g_v = coef exp2(s2_v - lse2) and,
// at entry k's id, q_k - p_k (entries with the same id hold the same sum).
struct VocabCoef {
    VocabRows r;
    const float *logq, *loss, *lse, *d_loss, *d_lse;
    float scale;
    float *lse2, *coef;  // [Np]
    float *at;           // [K][Np]: g at entry k's id
};

struct VocabJoin {
    VocabRows r;
    const float2* part;  // [parts][Np]: max, sum of exp2
    int parts;
    float2* state;       // [Np] of the pieces before, or NULL
    bool first, last;
    const float* slog;   // [K][Np] logits at the ids, times log2 e
    float *loss, *lse, *logq;
    uint32_t* err;       // for rows that are not listed
};
int launch_vocab_join(const VocabJoin& j, hipStream_t stream);

// Of the kernels before a product, those that wait for the list of rows alone, in one
// launch: any of packing h, turning h, the factors, and packing and turning W's piece.
struct VocabBegin {
    const VocabPack *pack_h = nullptr, *turn_h = nullptr, *pack_w = nullptr, *turn_w = nullptr;
    const VocabCoef* coef = nullptr;
};
int launch_vocab_begin(const VocabBegin& b, int dtype, hipStream_t stream);

// g at the entries' ids within the piece [v0, v0 + n).
struct VocabPatch {
    VocabRows r;
    const float* at;
    int v0, n, terms;
    int64_t ld_g, plane;
    uint16_t *g, *gt;  // [terms][Np][ld_g], [terms][piece][Np]
};
int launch_vocab_patch(const VocabPatch& p, hipStream_t stream);

// The parts of d_h's sum over the vocabulary: `parts` for n rows, and as many more (up to
// `most`) as the workgroups form that rows which are left out would have taken.
struct VocabSplit {
    const int32_t* count;
    int n, tile, parts, most;
    __device__ __forceinline__ int rows() const { return (min(n, *count) + tile - 1) / tile; }  // of tiles
    __device__ __forceinline__ int of(int rows) const {
        return max(min(parts * ((n + tile - 1) / tile) / max(rows, 1), most), 1);
    }
};

// The sum over parts [parts][part / Dp][Dp], in the caller's tensor.
struct VocabSum {
    const float* acc;
    int64_t part;
    int parts, Dp;
    VocabSplit split;    // with a count: it says the parts, of whole tiles of rows
    const int32_t* pos;  // d_h: where row i's sum is, kRowOut (zero) or kRowBad (NaN); NULL: at i
    int n, D;            // of out
    int dtype;
    void* out;
    int64_t ld;
    bool accumulate;
};
int launch_vocab_sum(const VocabSum& d, hipStream_t stream);

// out[n][m] = sum_k A[m][k] B[n][k] over planes of bf16 terms, k in steps of 64.
struct VocabGemm {
    const uint16_t *a, *b;
    int64_t a_plane, b_plane, lda, ldb;
    int m, n, k;           // rows of A and of B, and length of the sum (d_w: count's)
    const int32_t* count;  // device: bounds n (d_w: k, in whole steps)
    int64_t Np;
    // logits
    float scale2;          // scale * log2 e
    int v0, K;             // the piece's start, ids a row
    int64_t ld_g;          // g [terms][Np][ld_g], gt [terms][piece][Np]
    float2* part;          // forward
    const int32_t* kid;
    float* slog;
    const float *lse2, *coef;  // backward
    uint16_t *g, *gt;
    // gradients: parts of k, each of whole tiles of rows (d_h, f32 always: how many is
    // split's to say) or out_part values apart
    void* out;
    int64_t ld_out, out_part;
    VocabSplit split;
    int splits, out_dtype;
    bool accumulate;
};
int vocab_parts(const VocabGemm& g, int terms);  // partials of a forward's logits, at most m / 64 + 4
int launch_vocab_logits_fwd(const VocabGemm& g, int terms, hipStream_t stream);
int launch_vocab_logits_bwd(const VocabGemm& g, int terms, hipStream_t stream);
// both products of the gradient (n = 0: not that one)
int launch_vocab_grads(const VocabGemm& d_h, const VocabGemm& d_w, int terms, bool big, hipStream_t stream);

// Up to 64 rows (Np = 64), h and W read where they lie.  Rows keep their places; one
// that is left out has pos < 0.
constexpr int kVocabFew = 64;
struct VocabFew {
    VocabRows r;
    const void *h, *w;
    int64_t ld_h, ld_w;
    const uint16_t* hp;    // f32: h's terms [3][Np][width rounded up to 64]
    float scale2;
    int v0, P;             // the piece
    float2* part;          // forward, a partial for every vocab_few_part of the piece
    float* slog;
    const float *lse2, *coef, *at;  // backward, as VocabCoef
    uint16_t *g, *gt;
    const uint16_t* ht;    // h turned
    void* d_w;             // of the piece, row stride ld_w
    int dw_dtype;
    bool accumulate;
    float* acc;            // d_h: [splits][Np][width rounded up to 64]
    int splits;
    bool first;            // the first piece: acc holds nothing yet
};
int vocab_few_part(const VocabRows& r);  // of the vocabulary a partial stands for
int vocab_few_splits(int64_t V, int64_t D);
int launch_vocab_few_logits(const VocabFew& p, bool backward, hipStream_t stream);
int launch_vocab_few_d_h(const VocabFew& p, hipStream_t stream);
int launch_vocab_few_d_w(const VocabFew& p, hipStream_t stream);
// Before the backward: pos, the factors, and h turned, [terms][width][Np], with the rows
// that are left out zero; in f32 also h's terms, packed.
int launch_vocab_few_begin(const VocabCoef& c, const VocabPack& turned, const VocabPack& packed, hipStream_t stream);

// Stores what no kernel of this launch reads again past the caches: the operands that
// its workgroups share stay there (the backward's logits of 16384 x 16384 rows, width
// 2560, take 1095 us, with plain stores 1220).  V may be aligned to its elements only.
template <typename E, typename V>
__device__ __forceinline__ void stream_out(E* to, const V& v) {
    constexpr int N = sizeof(V);
    static_assert(N == 8 || N == 16 || N == 32, "");
    typedef uint32_t Piece __attribute__((ext_vector_type(N == 8 ? 2 : 4), aligned(sizeof(E) < 4 ? 2 : 4)));
    constexpr int K = N == 32 ? 2 : 1;
    Piece w[K];
    __builtin_memcpy(w, &v, N);
#pragma unroll
    for (int x = 0; x < K; ++x) __builtin_nontemporal_store(w[x], reinterpret_cast<Piece*>(to) + x);
}

// Stores a lane's V neighbouring values of a row of d_w; `left` of them are there.
template <typename E, int V>
__device__ __forceinline__ void store_dw(E* to, float (&v)[V], int left, bool accumulate) {
#pragma unroll
    for (int r = 0; r < V; ++r)
        if (accumulate && r < left) v[r] += to_f32(to[r]);
    E w[V];
#pragma unroll
    for (int r = 0; r < V; ++r) store_io(&w[r], v[r]);
    if (left >= V) stream_out(to, w);
    else
#pragma unroll
        for (int r = 0; r < V; ++r)
            if (r < left) to[r] = w[r];
}

// Joins two partials of a softmax: a maximum, and the sum of exp2 of what is over it.
__device__ __forceinline__ void merge(float& m, float& s, float m2, float s2) {
    const float top = fmaxf(m, m2);
    // an infinite sum stays one whatever it is scaled by
    s = (s < __builtin_inff() ? s * fast_exp2(m - top) : s) + (s2 < __builtin_inff() ? s2 * fast_exp2(m2 - top) : s2);
    m = top;
}

// v's next bf16 term, of TERMS in all; v keeps the rest.  One: v rounded.  Two: that,
// and the rest rounded (2^-17 of v is left).  Three: v itself, each term what the ones
// before leave with the low half cut off, so that no rounding passes the largest
// value; an infinity leaves a NaN.
template <int TERMS>
__device__ __forceinline__ uint16_t next_term(float& v) {
    if constexpr (TERMS < 3) {
        const uint16_t t = bf16_rne(v);
        v = fabsf(to_f32(t)) < __builtin_inff() ? v - to_f32(t) : 0.0f;
        return t;
    } else {
        const uint32_t bits = __float_as_uint(v);
        v -= __uint_as_float(bits & 0xffff0000u);
        return bits >> 16;
    }
}
template <int TERMS>
__device__ __forceinline__ void bf16_terms(float v, uint16_t (&t)[TERMS]) {
#pragma unroll
    for (int n = 0; n < TERMS; ++n) t[n] = next_term<TERMS>(v);
}

}  // namespace ssm
