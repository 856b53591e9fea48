// The losses over a vocabulary for up to 64 rows (decoded tokens, a short batch):
// bound by W's bytes, so W goes from memory to registers as it lies, once for the
// logits and once for d_h, in its own type and alignment, and nothing of it is
// laid out again.  With so few rows a gradient may hang on a single rounded value of
// g, and the products wait for W's bytes: g has a second bf16 term, which takes the
// first's rounding (up to 2^-8 of a value) out of the result but for 2^-17.
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

// Eight of the same values of h as they lie (f32 reads its terms from the workspace, which
// every workgroup would have to form again).
__device__ __forceinline__ u32x4 load_h(const VocabFew& p, int n, int k) {
    const bf16_t* row = static_cast<const bf16_t*>(p.h) + (int64_t)n * p.ld_h;
    u32x4 f;
    if (k + 8 <= p.r.D) {
        __builtin_memcpy(&f, row + k, 16);
    } else {
        bf16_t v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = k + e < p.r.D ? row[k + e] : 0;
        __builtin_memcpy(&f, v, 16);
    }
    return f;
}

// ---- the logits -----------------------------------------------------------------
// A group of KW waves has the sums of its 16 of the vocabulary from m0 of the piece in
// `red`, in KW parts.  Forward: a partial for the workgroup, and the logits at the rows'
// ids; backward: g in both orders.
constexpr int kM = 16, kRow = kM + 4;
template <int T, int NT, int KW, bool BWD>
__device__ __forceinline__ void finish(const VocabFew& p, float (&red)[KW][16 * NT][kRow], int m0) {
    constexpr int M = kM, N = 16 * NT, kLanes = 64 * KW / N, LPT = kLanes < M ? kLanes : M, VPT = M / LPT;
    constexpr int kGroups = 8 / KW;
    const VocabRows& r = p.r;
    const int group = threadIdx.x / (64 * KW), tid = threadIdx.x % (64 * KW);
    __shared__ float2 joined[kGroups][N];  // forward
    // LPT lanes of a wave share a row, with every LPT-th of its logits each
    const int n = tid / LPT, l = tid % LPT;
    const int there = min(M, r.V - p.v0 - m0);  // of the vocabulary: none or less past its end
    const bool work = n < N && m0 < p.P;  // whole waves; a group may lie past the piece
    if (work) {
        float s2[VPT];
#pragma unroll
        for (int x = 0; x < VPT; ++x) {
            float s = 0.0f;
#pragma unroll
            for (int y = 0; y < KW; ++y) s += red[y][n][l + LPT * x];
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
            if (l == 0) joined[group][n] = make_float2(none ? -0x1p127f : m, s);
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
    if constexpr (!BWD) {
        __syncthreads();
        if (threadIdx.x < N) {
            float2 all = joined[0][threadIdx.x];
#pragma unroll
            for (int g = 1; g < kGroups; ++g)  // of those that lie in the piece
                if (m0 - M * group + M * g < p.P) merge(all.x, all.y, joined[g][threadIdx.x].x, joined[g][threadIdx.x].y);
            p.part[(int64_t)blockIdx.x * r.Np + threadIdx.x] = all;
        }
    }
    if constexpr (BWD) {
        __syncthreads();
        constexpr int GT = T == 3 ? 3 : 2;
        const int64_t plane = (int64_t)r.Np * p.P;
        if (work) {
            uint16_t g[VPT][GT];
#pragma unroll
            for (int x = 0; x < VPT; ++x) bf16_terms<GT>(red[0][n][VPT * l + x], g[x]);
#pragma unroll
            for (int t = 0; t < GT; ++t)
                __builtin_memcpy(p.g + t * plane + (int64_t)n * p.P + m0 + VPT * l, [&] {
                    struct { uint16_t v[VPT]; } o;
#pragma unroll
                    for (int x = 0; x < VPT; ++x) o.v[x] = g[x][t];
                    return o;
                }().v, 2 * VPT);
        }
        for (int x = tid; x < M * 8 && m0 < p.P; x += 64 * KW) {  // 8 rows of a column
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

// A workgroup of 8 waves owns 8 / KW groups of 16 of the vocabulary and all rows (16 NT of
// them).  The KW waves of a group share out the width in chunks of 64, a lane reading 16
// neighbouring values of a row of W, so that four lanes take a 128-byte line (bf16), and
// add up through LDS.  Waves with the same part of the width share h's chunk through LDS,
// in pieces of 16 bytes swizzled by their row: 64 rows, width 2560, vocabulary 32000: 67
// us with h read by every wave, 35 so.  W's chunks and h's are read two steps ahead: more
// take the registers that two workgroups a compute unit have.
template <typename E, int NT, int KW, bool BWD>
__global__ __launch_bounds__(512, kTerms<E> == 1 ? 4 : 2) void few_logits(VocabFew p) {
    constexpr int T = kTerms<E>, N = 16 * NT, kStage = KW * T * N * 128, kRed = 8 * N * kRow * 4;
    constexpr int kPieces = KW * T * N * 8, X = (kPieces + 511) / 512, kAhead = 2;
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kStage > kRed ? 2 * kStage : kRed];
    const VocabRows& r = p.r;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane >> 4;
    const int i16 = lane & 15, group = wave / KW, part = wave % KW;
    const int m0 = (blockIdx.x * (8 / KW) + group) * 16;  // in the piece
    const E* w = static_cast<const E*>(p.w) + (int64_t)min(p.v0 + m0 + i16, r.V - 1) * p.ld_w;
    const int steps = (r.D + 64 * KW - 1) / (64 * KW);
    Raw<E> ring[kAhead];
    u32x4 hold[kAhead][X];
    auto fetch = [&](int s, Raw<E>& a, u32x4 (&h)[X]) {
#pragma unroll
        for (int x = 0; x < X; ++x) {
            const int at = threadIdx.x + 512 * x, n = min(at / 8 % N, r.N - 1), t = at / (8 * N) % T;
            const int k = 64 * (s * KW + at / (8 * N * T)) + 8 * (at % 8);
            if (kPieces % 512 && at >= kPieces) continue;
            if constexpr (T == 1) {
                h[x] = load_h(p, n, k);
            } else {
                const int64_t Kd = (r.D + 63) / 64 * 64;
                h[x] = k < Kd ? *reinterpret_cast<const u32x4*>(p.hp + (t * r.Np + n) * Kd + k) : u32x4{0, 0, 0, 0};
            }
        }
        a.load(w, 64 * (s * KW + part) + 16 * q, r.D);
    };
    auto put = [&](const u32x4 (&h)[X], uint8_t* to) {
#pragma unroll
        for (int x = 0; x < X; ++x) {
            const int at = threadIdx.x + 512 * x, row = at / 8;
            if (kPieces % 512 && at >= kPieces) continue;
            *reinterpret_cast<u32x4*>(to + row * 128 + 16 * ((at ^ row) & 7)) = h[x];
        }
    };
    f32x4 acc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        if (u < steps) fetch(u, ring[u], hold[u]);
    put(hold[0], lds);
    __syncthreads();
    for (int s0 = 0; s0 < steps; s0 += kAhead)
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int s = s0 + u;
            if (s < steps) {
                if (s + 1 < steps) put(hold[(u + 1) % kAhead], lds + (u + 1) % 2 * kStage);
                const Raw<E> cur = ring[u];
                if (s + kAhead < steps) fetch(s + kAhead, ring[u], hold[u]);
                const uint8_t* from = lds + u % 2 * kStage + part * (T * N * 128);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    u32x4 a[T], x[T][NT];
                    cur.operand(half, a);
#pragma unroll
                    for (int t = 0; t < T; ++t)
#pragma unroll
                        for (int j = 0; j < NT; ++j)
                            x[t][j] = *reinterpret_cast<const u32x4*>(from + (t * N + 16 * j + i16) * 128 +
                                                                      16 * ((2 * q + half) ^ (i16 & 7)));
                    // products' order, rows by turns: no product waits for the one before it
#pragma unroll
                    for (int y = T == 1 ? 5 : 0; y < 6; ++y)
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            const int ta = (0x001102 >> (4 * y)) & 15, tb = (0x010120 >> (4 * y)) & 15;
                            acc[j] = mfma(a[ta], x[tb][j], acc[j]);
                        }
                }
                __syncthreads();
            }
        }
    float (&red)[KW][N][kRow] = reinterpret_cast<float (*)[KW][N][kRow]>(lds)[group];
#pragma unroll
    for (int j = 0; j < NT; ++j) *reinterpret_cast<f32x4*>(&red[part][16 * j + i16][4 * q]) = acc[j];
    __syncthreads();
    finish<T, NT, KW, BWD>(p, red, m0);
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
    // in bf16 g is read with W, a step ahead; in f32, where it takes more registers, ahead
    // of the splitting of W
    constexpr bool kAhead = T == 1;
    struct Step {
        uint32_t w[8][kWords];
        u32x4 g[NT][GT];
    } next;
    auto load_g = [&](Step& s, int step) {
        const int v = 32 * step + 8 * q;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int t = 0; t < GT; ++t) {
                // written to the end of a group's 16 of the vocabulary
                const u32x4 x = *reinterpret_cast<const u32x4*>(p.g + t * plane + (int64_t)(16 * j + i16) * p.P + v);
                s.g[j][t] = v < rows ? x : u32x4{0, 0, 0, 0};
            }
    };
    auto load = [&](Step& s, int step) {
        if constexpr (kAhead) load_g(s, step);
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
        Step cur = next;
        if constexpr (!kAhead) load_g(cur, s);
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
            for (int j = 0; j < NT; ++j) acc[t][j] = products<T, GT>(a, cur.g[j], acc[t][j]);
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
// A workgroup owns 256 columns and 64 of the vocabulary; the sum over the rows is one
// or two MFMAs long, and d_w's bytes bound it.  A wave forms 64 columns, 16 of the
// vocabulary at a time, and the results leave through LDS, so that a wave stores whole
// runs of a row: 2 rows, width 1314, vocabulary 86475: 207 us with 64-byte pieces of 16
// rows a store, 73 so.
template <typename E, int T, int KS>
__global__ __launch_bounds__(256, 2) void few_d_w(VocabFew p) {
    constexpr int GT = T == 3 ? 3 : 2, kV = 64, kD = 256, kChunk = 16 / sizeof(E);
    __shared__ __attribute__((aligned(16))) E tile[kV][kD + kChunk];
    const VocabRows& r = p.r;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4, i16 = lane & 15;
    const int d0 = kD * blockIdx.x, v0 = kV * blockIdx.y, rows = min(p.P, r.V - p.v0);
    u32x4 a[4][KS][T], b[kV / 16][KS][GT];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int n = 0; n < T; ++n)
                a[t][k][n] = *reinterpret_cast<const u32x4*>(
                    p.ht + ((int64_t)n * r.D + min(d0 + 64 * wave + 16 * t + i16, r.D - 1)) * r.Np + 32 * k + 8 * q);
    const int64_t plane = (int64_t)r.Np * p.P;
#pragma unroll
    for (int s = 0; s < kV / 16; ++s)
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int n = 0; n < GT; ++n)
                b[s][k][n] = r.N == 0 ? u32x4{0, 0, 0, 0}  // without rows nothing wrote it
                                      : *reinterpret_cast<const u32x4*>(
                                            p.gt + n * plane + (int64_t)min(v0 + 16 * s + i16, rows - 1) * r.Np +
                                            32 * k + 8 * q);
#pragma unroll
    for (int s = 0; s < kV / 16; ++s)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            f32x4 acc = {0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < KS; ++k) acc = products<T, GT>(a[t][k], b[s][k], acc);
            E o[4];
            // what is added to is added to in f32
            E* at = &tile[16 * s + i16][64 * wave + 16 * t + 4 * q];
            if (p.accumulate && v0 + 16 * s + i16 < rows) {
                const E* old = static_cast<const E*>(p.d_w) + (int64_t)(v0 + 16 * s + i16) * p.ld_w;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int d = d0 + 64 * wave + 16 * t + 4 * q + x;
                    if (d < r.D) acc[x] += to_f32(old[d]);
                }
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) store_io(&o[x], acc[x]);
            __builtin_memcpy(at, o, sizeof o);
        }
    __syncthreads();
    constexpr int kChunks = kD / kChunk;  // of a row
    for (int x = threadIdx.x; x < kV * kChunks; x += 256) {
        const int v = x / kChunks, c = x % kChunks * kChunk, left = r.D - d0 - c;
        if (v0 + v >= rows || left <= 0) continue;
        E* to = static_cast<E*>(p.d_w) + (int64_t)(v0 + v) * p.ld_w + d0 + c;
        const u32x4 w = *reinterpret_cast<const u32x4*>(&tile[v][c]);
        if (left >= kChunk) {
            stream_out(to, w);
        } else {
#pragma unroll
            for (int e = 0; e < kChunk; ++e)
                if (e < left) to[e] = tile[v][c + e];
        }
    }
}

// How the logits are shared out: 16 nt rows, and kw waves a group, more of them where the
// last round of workgroups then leaves fewer compute units idle.  (W from memory, bf16: 64
// rows, width 2560, vocabulary 32000: 72 us with 1, 54 with 2, 65 with 4; vocabulary 131072:
// 152, 172 and 220; 2 rows, width 1314, vocabulary 86475: 83, 66 and 70.)
struct FewTile {
    int nt, kw;
};
FewTile few_tile(const VocabRows& r) {
    FewTile f = {r.N <= 16 ? 1 : r.N <= 32 ? 2 : 4, 1};
    // 64 rows in f32: one workgroup a compute unit, and four waves a group take 192 KB of LDS
    const bool large = r.terms == 3 && f.nt == 4;
    const int64_t places = large ? 256 : 512;
    double best = 0.0;
    for (int kw = 1; kw <= (large ? 2 : 4); kw *= 2) {
        // a wave takes four steps at least unless most places are empty (15 rows, width 144,
        // vocabulary 77982: 22 us with 2, 15 with 1)
        if (kw > 1 && (best < 0.5 ? 32 : 256) * kw > r.D) break;
        const int64_t groups = ((int64_t)r.V * kw + 127) / 128, rounds = (groups + places - 1) / places;
        const double used = (double)groups / (rounds * places);
        if (used > 1.1 * best) {
            best = used;
            f.kw = kw;
        }
    }
    return f;
}

template <typename E, int NT, bool BWD>
void start(const VocabFew& p, int kw, int v, hipStream_t stream) {
    const unsigned grid = (v + 128 / kw - 1) / (128 / kw);
    if (kw == 1) few_logits<E, NT, 1, BWD><<<grid, 512, 0, stream>>>(p);
    else if (kw == 2) few_logits<E, NT, 2, BWD><<<grid, 512, 0, stream>>>(p);
    else if constexpr (sizeof(E) == 2 || NT < 4) few_logits<E, NT, 4, BWD><<<grid, 512, 0, stream>>>(p);
}

template <typename E, bool BWD>
int launch_logits(const VocabFew& p, hipStream_t stream) {
    const FewTile f = few_tile(p.r);
    const int v = p.r.V - p.v0 < p.P ? p.r.V - p.v0 : p.P;
    if (f.nt == 1) start<E, 1, BWD>(p, f.kw, v, stream);
    else if (f.nt == 2) start<E, 2, BWD>(p, f.kw, v, stream);
    else start<E, 4, BWD>(p, f.kw, v, stream);
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

template <bool BWD>
int launch_logits(const VocabFew& p, hipStream_t stream) {
    return p.r.terms == 3 ? launch_logits<float, BWD>(p, stream) : launch_logits<bf16_t, BWD>(p, stream);
}

template <typename E>
int launch_d_h(const VocabFew& p, hipStream_t stream) {
    const dim3 grid((p.r.D + 255) / 256, p.splits);
    const int nt = few_tile(p.r).nt;
    if (nt == 1) few_d_h<E, 1><<<grid, 256, 0, stream>>>(p);
    else if (nt == 2) few_d_h<E, 2><<<grid, 256, 0, stream>>>(p);
    else few_d_h<E, 4><<<grid, 256, 0, stream>>>(p);
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

template <typename E, int T>
int launch_d_w(const VocabFew& p, hipStream_t stream) {
    const int rows = p.r.V - p.v0 < p.P ? p.r.V - p.v0 : p.P;
    const dim3 grid((p.r.D + 255) / 256, (rows + 63) / 64);
    if (p.r.N <= 32) few_d_w<E, T, 1><<<grid, 256, 0, stream>>>(p);
    else few_d_w<E, T, 2><<<grid, 256, 0, stream>>>(p);
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // namespace

int vocab_few_part(const VocabRows& r) { return 128 / few_tile(r).kw; }

// Parts of d_h's sum over the vocabulary, of 4 steps at least: four workgroups a compute
// unit, and not many more, since every part is written and read again.
int vocab_few_splits(int64_t V, int64_t D) {
    const int64_t columns = (D + 255) / 256, most = (V + 127) / 128;
    int64_t n = 1024 / columns;
    if (n > most) n = most;
    return (int)(n < 1 ? 1 : n > 256 ? 256 : n);
}

int launch_vocab_few_logits(const VocabFew& p, bool backward, hipStream_t stream) {
    return backward ? launch_logits<true>(p, stream) : launch_logits<false>(p, stream);
}

int launch_vocab_few_d_h(const VocabFew& p, hipStream_t stream) {
    return p.r.terms == 3 ? launch_d_h<float>(p, stream) : launch_d_h<bf16_t>(p, stream);
}

int launch_vocab_few_d_w(const VocabFew& p, hipStream_t stream) {
    if (p.r.terms == 3) return launch_d_w<float, 3>(p, stream);
    return p.dw_dtype == SSM_F32 ? launch_d_w<float, 1>(p, stream) : launch_d_w<bf16_t, 1>(p, stream);
}

}  // namespace ssm
