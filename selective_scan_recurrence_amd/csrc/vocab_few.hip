// The losses over a vocabulary for up to 64 rows (decoded tokens, a short batch):
// bound by W's bytes, so W goes from memory to registers as it lies, once for the
// logits and once for d_h, in its own type and alignment, and nothing of it is
// laid out again.
#include <type_traits>

#include "vocab.h"

namespace ssm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

// sums of the products of terms that count, small ones first
template <int TA, int TB>
__device__ __forceinline__ f32x4 products(const u32x4 (&a)[TA], const u32x4 (&b)[TB], f32x4 c) {
    if constexpr (TA == 3 && TB == 3) {
        c = mfma(a[2], b[0], c);
        c = mfma(a[0], b[2], c);
        c = mfma(a[1], b[1], c);
        c = mfma(a[1], b[0], c);
        c = mfma(a[0], b[1], c);
    } else {
#pragma unroll
        for (int n = TB - 1; n > 0; --n) c = mfma(a[0], b[n], c);
    }
    return mfma(a[0], b[0], c);
}

template <typename E>
constexpr int kTerms = std::is_same<E, bf16_t>::value ? 1 : 3;

// Sixteen values of a row as they lie, and as operands: MFMA h takes values 8 h ..
// 8 h + 7 of every lane (which k a lane's values are does not matter as long as
// both operands agree).
template <typename E>
struct Raw {
    static constexpr int kWords = sizeof(E) * 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const E* row, int k, int width) {
        if (k + 16 <= width) {
            __builtin_memcpy(w, row + k, sizeof w);
            return;
        }
        E v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = k + e < width ? row[k + e] : E(0);
        __builtin_memcpy(w, v, sizeof w);
    }
    __device__ __forceinline__ void operand(int h, u32x4 (&f)[kTerms<E>]) const {
        if constexpr (kTerms<E> == 1) {
            f[0] = u32x4{w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]};
        } else {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                uint16_t a[3], b[3];
                bf16_terms<3>(__uint_as_float(w[8 * h + 2 * p]), a);
                bf16_terms<3>(__uint_as_float(w[8 * h + 2 * p + 1]), b);
#pragma unroll
                for (int n = 0; n < 3; ++n) f[n][p] = a[n] | (uint32_t)b[n] << 16;
            }
        }
    }
};

// The same sixteen values of h: as they lie, or (f32) of its terms in the workspace,
// which every workgroup would have to form again.
template <typename E>
struct Rows {
    Raw<E> x;
    __device__ __forceinline__ void load(const VocabFew& p, int n, int k) {
        x.load(static_cast<const E*>(p.h) + (int64_t)n * p.ld_h, k, p.r.D);
    }
    __device__ __forceinline__ void operand(int h, u32x4 (&f)[1]) const { x.operand(h, f); }
};
template <>
struct Rows<float> {
    u32x4 x[2][3];
    __device__ __forceinline__ void load(const VocabFew& p, int n, int k) {
        const int64_t Kd = (p.r.D + 63) / 64 * 64;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < 3; ++t)
                x[h][t] = *reinterpret_cast<const u32x4*>(p.hp + (t * p.r.Np + n) * Kd + k + 8 * h);
    }
    __device__ __forceinline__ void operand(int h, u32x4 (&f)[3]) const {
#pragma unroll
        for (int t = 0; t < 3; ++t) f[t] = x[h][t];
    }
};

// ---- the logits -----------------------------------------------------------------
// A workgroup of 8 waves owns 16 MT of the vocabulary and all rows (16 NT of them).
// The waves share out the width in chunks of 64, a lane reading 16 neighbouring
// values of a row, so that four lanes take a 128-byte line (bf16), and add up
// through LDS.
template <typename E, int MT, int NT, bool BWD>
__global__ __launch_bounds__(512, 2) void few_logits(VocabFew p) {
    constexpr int T = kTerms<E>, M = 16 * MT, N = 16 * NT, LPT = 512 / N < M ? 512 / N : M, VPT = M / LPT, kRow = M + 4;
    __shared__ __attribute__((aligned(16))) float red[8][N][kRow];
    const VocabRows& r = p.r;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, q = lane >> 4, i16 = lane & 15;
    const int m0 = blockIdx.x * M;  // in the piece
    const E* w[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
        w[t] = static_cast<const E*>(p.w) + (int64_t)min(p.v0 + m0 + 16 * t + i16, r.V - 1) * p.ld_w;
    f32x4 acc[MT][NT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[t][j] = f32x4{0, 0, 0, 0};
    Raw<E> next[MT];
    int k = 64 * wave + 16 * q;
    if (64 * wave < r.D)
#pragma unroll
        for (int t = 0; t < MT; ++t) next[t].load(w[t], k, r.D);
    for (; k - 16 * q < r.D; k += 512) {
        Raw<E> cur[MT];
        Rows<E> x[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) x[j].load(p, min(16 * j + i16, r.N - 1), k);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            cur[t] = next[t];
            if (k - 16 * q + 512 < r.D) next[t].load(w[t], k + 512, r.D);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            u32x4 b[NT][T];
#pragma unroll
            for (int j = 0; j < NT; ++j) x[j].operand(half, b[j]);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                u32x4 a[T];
                cur[t].operand(half, a);
#pragma unroll
                for (int j = 0; j < NT; ++j) acc[t][j] = products<T, T>(a, b[j], acc[t][j]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            *reinterpret_cast<f32x4*>(&red[wave][16 * j + i16][16 * t + 4 * q]) = acc[t][j];
    __syncthreads();

    // LPT lanes of a wave share a row, with every LPT-th of its logits each
    const int n = tid / LPT, l = tid % LPT;
    const int there = min(M, r.V - p.v0 - m0);  // of the vocabulary
    if (n < N) {  // whole waves
        float s2[VPT];
#pragma unroll
        for (int x = 0; x < VPT; ++x) {
            float s = 0.0f;
#pragma unroll
            for (int y = 0; y < 8; ++y) s += red[y][n][l + LPT * x];
            s2[x] = s * p.scale2;
        }
        if constexpr (!BWD) {
            float m = -__builtin_inff();
#pragma unroll
            for (int x = 0; x < VPT; ++x) {
                if (l + LPT * x >= there) s2[x] = -__builtin_inff();
                m = fmaxf(m, s2[x]);
            }
#pragma unroll
            for (int d = 1; d < LPT; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
            // as the tiles' statistics: nothing is taken off an infinite maximum
            const bool none = !(m > -__builtin_inff());
            m = fabsf(m) < __builtin_inff() ? m : 0.0f;
            float s = 0.0f;
#pragma unroll
            for (int x = 0; x < VPT; ++x) s += fast_exp2(s2[x] - m);
#pragma unroll
            for (int d = 1; d < LPT; d *= 2) s += __shfl_xor(s, d);
            if (l == 0) p.part[(int64_t)blockIdx.x * r.Np + n] = make_float2(none ? -0x1p127f : m, s);
        } else {
            const bool out = n >= r.N || r.pos[n] < 0;
            const float a = out ? 0.0f : p.coef[n], lse2 = out ? 0.0f : p.lse2[n];
#pragma unroll
            for (int x = 0; x < VPT; ++x)
                s2[x] = out || l + LPT * x >= there ? 0.0f : a * fast_exp2(s2[x] - lse2);
        }
        // a lane's own sums give way to the results
#pragma unroll
        for (int x = 0; x < VPT; ++x) red[0][n][l + LPT * x] = s2[x];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (n < r.N)
            for (int y = l; y < r.K; y += LPT) {
                const int64_t e = (int64_t)n * r.K + y;
                const int id = r.id[e], at = id - p.v0 - m0;
                if (id < p.v0 + m0 || at >= there || (r.logit && r.logit[e] == -__builtin_inff())) continue;
                if constexpr (!BWD) p.slog[(int64_t)y * r.Np + n] = red[0][n][at];
                else if (r.pos[n] >= 0) red[0][n][at] = p.at[(int64_t)y * r.Np + n];
            }
    }
    if constexpr (BWD) {
        __syncthreads();
        constexpr int GT = T == 3 ? 3 : 2;
        const int64_t plane = (int64_t)r.Np * p.P;
        if (n < N) {
            uint16_t g[VPT][GT];
#pragma unroll
            for (int x = 0; x < VPT; ++x) bf16_terms<GT>(red[0][n][VPT * l + x], g[x]);
#pragma unroll
            for (int t = 0; t < GT; ++t)
#pragma unroll
                for (int x = 0; x < VPT; ++x) p.g[t * plane + (int64_t)n * p.P + m0 + VPT * l + x] = g[x][t];
        }
        for (int x = tid; x < M * 8; x += 512) {  // 8 rows of one column
            const int m = x / 8, n0 = x % 8 * 8;
            uint16_t v[8][GT];
#pragma unroll
            for (int e = 0; e < 8; ++e) bf16_terms<GT>(n0 + e < N ? red[0][min(n0 + e, N - 1)][m] : 0.0f, v[e]);
#pragma unroll
            for (int t = 0; t < GT; ++t) {
                u32x4 o;
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = v[2 * e][t] | (uint32_t)v[2 * e + 1][t] << 16;
                *reinterpret_cast<u32x4*>(p.gt + t * plane + (int64_t)(m0 + m) * r.Np + n0) = o;
            }
        }
    }
}

// ---- d_h ------------------------------------------------------------------------
// A wave owns 64 columns and a part of the vocabulary, 32 of it a step: lane 16 q + i
// reads columns 4 i .. 4 i + 3 of the rows 8 q .. 8 q + 7 of W and pairs rows with a
// byte permute a register; its four columns belong to four MFMA tiles.
template <typename E, int NT>
__global__ __launch_bounds__(256, 2) void few_d_h(VocabFew p) {
    constexpr int T = kTerms<E>, GT = T == 3 ? 3 : 2, kWords = sizeof(E);
    const VocabRows& r = p.r;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4, i16 = lane & 15;
    const int d0 = 256 * blockIdx.x + 64 * wave, col = d0 + 4 * i16;
    if (d0 >= r.D) return;
    const int rows = min(p.P, r.V - p.v0), steps = (rows + 31) / 32;
    const int begin = (int)((int64_t)steps * blockIdx.y / p.splits), end = (int)((int64_t)steps * (blockIdx.y + 1) / p.splits);
    const E* w = static_cast<const E*>(p.w) + (int64_t)p.v0 * p.ld_w;
    const int64_t plane = (int64_t)r.Np * p.P;
    f32x4 acc[4][NT];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[t][j] = f32x4{0, 0, 0, 0};
    struct Step {
        uint32_t w[8][kWords];
    } next;
    auto load = [&](Step& s, int step) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // g is zero past the vocabulary
            const E* row = w + (int64_t)min(32 * step + 8 * q + j, rows - 1) * p.ld_w;
            if (col + 4 <= r.D) {
                __builtin_memcpy(s.w[j], row + col, sizeof s.w[j]);
            } else {
                E x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = col + e < r.D ? row[col + e] : E(0);
                __builtin_memcpy(s.w[j], x, sizeof x);
            }
        }
    };
    if (begin < end) load(next, begin);
    for (int s = begin; s < end; ++s) {
        const Step cur = next;
        u32x4 g[NT][GT];
        const int v = 32 * s + 8 * q;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int t = 0; t < GT; ++t) {
                // written to the end of a workgroup's 16 MT of the vocabulary
                const u32x4 x = *reinterpret_cast<const u32x4*>(p.g + t * plane + (int64_t)(16 * j + i16) * p.P + v);
                g[j][t] = v < rows ? x : u32x4{0, 0, 0, 0};
            }
        if (s + 1 < end) load(next, s + 1);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            u32x4 a[T];
            if constexpr (T == 1) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    a[0][x] = __builtin_amdgcn_perm(cur.w[2 * x + 1][t / 2], cur.w[2 * x][t / 2],
                                                    t & 1 ? 0x07060302u : 0x05040100u);
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint16_t u[3], y[3];
                    bf16_terms<3>(__uint_as_float(cur.w[2 * x][t]), u);
                    bf16_terms<3>(__uint_as_float(cur.w[2 * x + 1][t]), y);
#pragma unroll
                    for (int n = 0; n < 3; ++n) a[n][x] = u[n] | (uint32_t)y[n] << 16;
                }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[t][j] = products<T, GT>(a, g[j], acc[t][j]);
        }
    }
    // tile t's row 4 q + x is column 4 (4 q + x) + t: 16 neighbours a lane
    const int64_t Dp = (r.D + 63) / 64 * 64;
    float* out = p.acc + (int64_t)blockIdx.y * r.Np * Dp;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const f32x4 v = {acc[0][j][x], acc[1][j][x], acc[2][j][x], acc[3][j][x]};
            f32x4* to = reinterpret_cast<f32x4*>(out + (int64_t)(16 * j + i16) * Dp + d0 + 16 * q + 4 * x);
            *to = p.first ? v : *to + v;
        }
}

// ---- d_w ------------------------------------------------------------------------
// A wave owns 64 columns and 128 of the vocabulary, 16 of it a step; the sum over the
// rows is one or two MFMAs long, and d_w's bytes bound it.  Tiles take the columns in
// the order of the big products' rows (S neighbouring groups of 4 a lane).
template <int T, int KS, int S>
__global__ __launch_bounds__(256, 2) void few_d_w(VocabFew p) {
    constexpr int GT = T == 3 ? 3 : 2, kSteps = 8;
    const VocabRows& r = p.r;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4, i16 = lane & 15;
    const int d0 = 256 * blockIdx.x + 64 * wave, rows = min(p.P, r.V - p.v0);
    if (d0 >= r.D) return;
    u32x4 a[4][KS][T];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int n = 0; n < T; ++n) {
                const int d = min(d0 + 16 * S * (t / S) + 4 * S * (i16 >> 2) + 4 * (t % S) + (i16 & 3), r.D - 1);
                a[t][k][n] = *reinterpret_cast<const u32x4*>(p.ht + ((int64_t)n * r.D + d) * r.Np + 32 * k + 8 * q);
            }
    const int64_t plane = (int64_t)r.Np * p.P;
    u32x4 next[KS][GT];
    auto load = [&](int v) {  // gt has a piece's rows, whole tiles of them
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int n = 0; n < GT; ++n)
                next[k][n] = r.N == 0 ? u32x4{0, 0, 0, 0}  // without rows nothing wrote it
                                      : *reinterpret_cast<const u32x4*>(p.gt + n * plane + (int64_t)(v + i16) * r.Np +
                                                                        32 * k + 8 * q);
    };
    const int begin = 16 * kSteps * blockIdx.y, end = min(begin + 16 * kSteps, rows);
    load(begin);
    for (int v = begin; v < end; v += 16) {
        u32x4 b[KS][GT];
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int n = 0; n < GT; ++n) b[k][n] = next[k][n];
        if (v + 16 < end) load(v + 16);
#pragma unroll
        for (int t = 0; t < 4; t += S) {
            float c[4 * S];
#pragma unroll
            for (int s = 0; s < S; ++s) {
                f32x4 acc = {0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < KS; ++k) acc = products<T, GT>(a[t + s][k], b[k], acc);
#pragma unroll
                for (int x = 0; x < 4; ++x) c[4 * s + x] = acc[x];
            }
            const int d = d0 + 16 * t + 4 * S * q, left = r.D - d;
            if (v + i16 >= rows || left <= 0) continue;
            const int64_t at = (int64_t)(v + i16) * p.ld_w + d;
            if (p.dw_dtype == SSM_F32) store_dw(static_cast<float*>(p.d_w) + at, c, left, p.accumulate);
            else store_dw(static_cast<bf16_t*>(p.d_w) + at, c, left, p.accumulate);
        }
    }
}

template <typename E, int MT, bool BWD>
int launch_logits(const VocabFew& p, hipStream_t stream) {
    const int M = 16 * MT, v = p.r.V - p.v0 < p.P ? p.r.V - p.v0 : p.P, grid = (v + M - 1) / M;
    if (p.r.N <= 16) few_logits<E, MT, 1, BWD><<<grid, 512, 0, stream>>>(p);
    else if (p.r.N <= 32) few_logits<E, MT, 2, BWD><<<grid, 512, 0, stream>>>(p);
    else if constexpr (MT < 4) few_logits<E, MT, 4, BWD><<<grid, 512, 0, stream>>>(p);  // 64 logits a workgroup are for up to 32 rows
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

template <bool BWD>
int launch_logits(const VocabFew& p, hipStream_t stream) {
    const int mt = vocab_few_tile(p.r.V, p.r.N, p.r.terms) / 16;
    if (p.r.terms == 3)
        return mt == 1 ? launch_logits<float, 1, BWD>(p, stream) : launch_logits<float, 2, BWD>(p, stream);
    return mt == 1   ? launch_logits<bf16_t, 1, BWD>(p, stream)
           : mt == 2 ? launch_logits<bf16_t, 2, BWD>(p, stream)
                     : launch_logits<bf16_t, 4, BWD>(p, stream);
}

}  // namespace

// Of the vocabulary a workgroup: the more, the fewer times h is read, as long as
// there is more than one workgroup a compute unit.
int vocab_few_tile(int64_t V, int N, int terms) {
    const int most = terms == 3 || N > 32 ? 32 : 64;
    int m = 16;
    while (m < most && V / (2 * m) >= 400) m *= 2;
    return m;
}

// Parts of d_h's sum over the vocabulary, of 4 steps at least: two workgroups a compute
// unit, and not many more, since every part is written and read again.
int vocab_few_splits(int64_t V, int64_t D) {
    const int64_t columns = (D + 255) / 256, most = (V + 127) / 128;
    int64_t n = 640 / columns;
    if (n > most) n = most;
    return (int)(n < 1 ? 1 : n > 256 ? 256 : n);
}

int launch_vocab_few_logits(const VocabFew& p, bool backward, hipStream_t stream) {
    return backward ? launch_logits<true>(p, stream) : launch_logits<false>(p, stream);
}

int launch_vocab_few_d_h(const VocabFew& p, hipStream_t stream) {
    const dim3 grid((p.r.D + 255) / 256, p.splits);
    const int nt = p.r.N <= 16 ? 1 : p.r.N <= 32 ? 2 : 4;
    if (p.r.terms == 3) {
        if (nt == 1) few_d_h<float, 1><<<grid, 256, 0, stream>>>(p);
        else if (nt == 2) few_d_h<float, 2><<<grid, 256, 0, stream>>>(p);
        else few_d_h<float, 4><<<grid, 256, 0, stream>>>(p);
    } else {
        if (nt == 1) few_d_h<bf16_t, 1><<<grid, 256, 0, stream>>>(p);
        else if (nt == 2) few_d_h<bf16_t, 2><<<grid, 256, 0, stream>>>(p);
        else few_d_h<bf16_t, 4><<<grid, 256, 0, stream>>>(p);
    }
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int launch_vocab_few_d_w(const VocabFew& p, hipStream_t stream) {
    const int rows = p.r.V - p.v0 < p.P ? p.r.V - p.v0 : p.P;
    const dim3 grid((p.r.D + 255) / 256, (rows + 127) / 128);
    const bool two = p.r.N > 32, f32 = p.dw_dtype == SSM_F32;
    if (p.r.terms == 3) {
        if (two) few_d_w<3, 2, 1><<<grid, 256, 0, stream>>>(p);
        else few_d_w<3, 1, 1><<<grid, 256, 0, stream>>>(p);
    } else if (f32) {
        if (two) few_d_w<1, 2, 1><<<grid, 256, 0, stream>>>(p);
        else few_d_w<1, 1, 1><<<grid, 256, 0, stream>>>(p);
    } else {
        if (two) few_d_w<1, 2, 2><<<grid, 256, 0, stream>>>(p);
        else few_d_w<1, 1, 2><<<grid, 256, 0, stream>>>(p);
    }
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // namespace ssm
