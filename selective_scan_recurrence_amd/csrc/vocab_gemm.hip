// The products of the losses over a vocabulary: out[n][m] = sum_k A[m][k] B[n][k],
// both operands with k fastest, in bf16 on MFMA with f32 sums.
//   logits:  A = W (m: vocabulary), B = h (n: rows);  forward: the softmax
//            statistics of each row over the tile's vocabulary, and the logits at
//            the row's ids; backward: g = coef exp2(s - lse), stored in both
//            orders, since one product sums over the vocabulary and one over rows
//   d_h:     A = W turned (m: width),  B = g (n: rows)
//   d_w:     A = h turned (m: width),  B = g turned (n: vocabulary)
// An f32 value is three bf16 terms, and a product the six largest of its nine partial
// products (the other three reach 2^-21 of it together), the small ones first: six runs
// over k.
//
// A workgroup of 2 x 2 waves owns 256 x 256 (or 128 x 128) of out and walks k in
// steps of 64: 128-byte rows go from memory to LDS past the registers, into one of
// two buffers while the other is multiplied.  LDS holds the rows in the order of
// MFMA tiles, row i (of 16) of tile t at 16 t + i, its 16-byte piece c at
// c ^ (i % 8): a read of operands then meets no bank twice.  Which row of A is row i
// of tile t is free: S tiles share 16 S rows, so that a lane (q = lane / 16, i = lane
// % 16) ends with 4 S neighbouring m from 4 S q.  S = 2 where they leave in bf16, 1
// in f32: the 4 lanes of a row of out then store 64 neighbouring bytes (with 16 m a
// lane, which leave in two stores of every second 16 bytes, the backward's logits of
// 16384 x 16384 rows, width 2560, took 1340 us, so 1220, and past the caches 1095).
// Tile j of a wave's TN tiles of B takes the rows TN i + j: TN neighbouring n a lane
// for g's other order.
//
// The big tile has one wave a SIMD with 64 accumulators of 4 registers each, a
// quarter fewer bytes from LDS than eight waves of 128 x 64.  That counts because
// the card's power bounds the loop: eight waves take 2959 cycles a step at 1.9 GHz
// and four 2775 at a lower clock, both 1.48 us, as a large library product does.
#include <type_traits>

#include "vocab.h"

namespace ssm {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void* lds_ptr;

constexpr std::true_type yes{};
constexpr std::false_type no{};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* base) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, 0xffffffff, 0x00020000);
}

// 16 bytes a lane from memory to LDS at `to` + 16 lane.  (The host's compiler does
// not know the builtin, and would drop the kernels that use it in a template.)
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t from, uint8_t* to, uint32_t lane_at, int at) {
#ifdef __HIP_DEVICE_COMPILE__
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_ptr)to, 16, lane_at, at, 0, 0);
#endif
}

// c += A B, with c in the accumulation registers: left to itself the compiler
// moves accumulators between the two halves of a 512-register wave.
__device__ __forceinline__ void mfma(f32x4& c, const u32x4& a, const u32x4& b) {
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}

// The waits between these and other uses of the accumulators, which the compiler
// does not see: 18 cycles are the most that a result of this size takes.
template <int TM, int TN>
__device__ __forceinline__ void settle(f32x4 (&c)[TM][TN]) {
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int j = 0; j < TN; j += 4)
            asm volatile("s_nop 0" : "+a"(c[t][j]), "+a"(c[t][j + 1]), "+a"(c[t][j + 2]), "+a"(c[t][j + 3]));
    asm volatile("s_nop 15" ::: "memory");
}

// The accumulators are read where they are used, not all of them before: they take
// half of the registers.
__device__ __forceinline__ f32x4 take(const f32x4& c) {
    f32x4 v;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v[0]) : "a"(c[0]));
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v[1]) : "a"(c[1]));
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v[2]) : "a"(c[2]));
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v[3]) : "a"(c[3]));
    return v;
}

// A run's planes.  Six runs: the partial products of three terms, small ones first.
template <int RUNS>
__device__ __forceinline__ int plane_a(int run) {
    return RUNS == 6 ? (0x001102 >> (4 * run)) & 15 : 0;
}
template <int RUNS>
__device__ __forceinline__ int plane_b(int run) {
    return RUNS == 6 ? (0x010120 >> (4 * run)) & 15 : 0;
}

// Tiles of out, numbered in bands of 8 columns.
struct Place {
    int mt, nt;
    __device__ __forceinline__ void of(int id, int* m, int* n) const {
        const int band = id / (mt * 8), in = id - band * mt * 8, wide = min(8, nt - 8 * band);
        *m = in / wide;
        *n = 8 * band + in % wide;
    }
};

// Workgroups are dealt to the 8 XCDs in turn: an XCD takes neighbouring tiles,
// which share A and B.  `pid` counts from the first of these tiles' workgroups.
// -1: no tile is left.
__host__ __device__ __forceinline__ int64_t on_xcds(int64_t total) { return (total + 7) / 8 * 8; }
__device__ __forceinline__ int tile_of(int pid, int total) {
    const int per = (total + 7) / 8, id = pid % 8 * per + pid / 8;
    return pid / 8 < per && id < total ? id : -1;
}

template <int TM_, int TN_>
struct Tile {
    static constexpr int WM = 2, WN = 2, NW = 4, TM = TM_, TN = TN_, BM = WM * TM * 16, BN = WN * TN * 16;
    static constexpr int kStage = (BM + BN) * 128;
    // two stages; the logits at the ids pass through 64 x TN 16 values a wave
    static constexpr int kLds = 2 * kStage;
    static_assert(NW * TN * 4096 <= kLds && TN % 4 == 0, "");
    static constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;
};
using Big = Tile<8, 8>;
using Small = Tile<4, 4>;

// Row i of tile t among a wave's rows of A.
template <int S>
__device__ __forceinline__ constexpr int row_of_a(int t, int i) {
    return 16 * S * (t / S) + 4 * S * (i >> 2) + 4 * (t % S) + (i & 3);
}

// acc = A[m0 ..] B[n0 ..]^T over steps [s0, s1) of every run.
template <class T, int RUNS, int S>
__device__ __forceinline__ void product(const VocabGemm& p, int m0, int n0, int n_rows, int s0, int s1, uint8_t* lds,
                                        f32x4 (&acc)[T::TM][T::TN]) {
    constexpr int TM = T::TM, TN = T::TN, LA = T::LA, LB = T::LB, NW = T::NW, kStage = T::kStage;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / T::WN, wn = wave % T::WN, q = lane >> 4, i16 = lane & 15;
    const int steps = s1 - s0, total = RUNS * steps;

    // a wave's load is half an MFMA tile, 8 rows of 8 pieces
    uint32_t at_a[LA], at_b[LB];
#pragma unroll
    for (int x = 0; x < LA; ++x) {
        const int l = 8 * (wave + NW * x) + lane / 8, t = l / 16, i = l % 16;
        at_a[x] = (uint32_t)min(row_of_a<S>(t, i), p.m - 1 - m0) * (uint32_t)(2 * p.lda) + 16 * ((lane & 7) ^ (i & 7));
    }
#pragma unroll
    for (int x = 0; x < LB; ++x) {
        const int l = 8 * (wave + NW * x) + lane / 8, t = l / 16, i = l % 16, row = 16 * TN * (t / TN) + TN * i + t % TN;
        at_b[x] = (uint32_t)min(row, n_rows - 1 - n0) * (uint32_t)(2 * p.ldb) + 16 * ((lane & 7) ^ (i & 7));
    }
    const uint16_t* a = p.a + (int64_t)m0 * p.lda + (int64_t)s0 * kVocabStep;
    const uint16_t* b = p.b + (int64_t)n0 * p.ldb + (int64_t)s0 * kVocabStep;
    __amdgpu_buffer_rsrc_t ra, rb;
    uint8_t* l_buf;
    int l_at;
    auto load_begin = [&](int step, uint8_t* buf) {
        const int run = RUNS == 1 ? 0 : step / steps, s = step - run * steps;
        ra = rsrc_of(a + plane_a<RUNS>(run) * p.a_plane);
        rb = rsrc_of(b + plane_b<RUNS>(run) * p.b_plane);
        l_buf = buf;
        l_at = s * (2 * kVocabStep);
    };
    auto load_one = [&](int x) {
        if (x < LA) load_lds(ra, l_buf + (wave + NW * x) * 1024, at_a[x], l_at);
        else load_lds(rb, l_buf + T::BM * 128 + (wave + NW * (x - LA)) * 1024, at_b[x - LA], l_at);
    };

#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[t][j] = f32x4{0, 0, 0, 0};
    settle(acc);

    // Row e = ks TM + t of a step multiplies A's tile t with B's TN tiles.  A's tiles
    // are read three rows ahead into a ring of four, B's of the next half step
    // during the half before.  Three rows before a step's end all of it has been
    // read: there every wave waits for the next step's loads, and begins those of
    // the step after it, two a row.
    const uint32_t row_a = (wm * TM * 16 + i16) * 128, row_b = (T::BM + wn * TN * 16 + i16) * 128;
    u32x4 fa[4], fb[2][TN];
    auto read_a = [&](int e, const uint8_t* buf) {
        fa[e & 3] = *reinterpret_cast<const u32x4*>(buf + row_a + (e % TM) * 2048 + 16 * ((4 * (e / TM) + q) ^ (i16 & 7)));
    };
    auto read_b = [&](int ks, int j, const uint8_t* buf) {
        fb[ks][j] = *reinterpret_cast<const u32x4*>(buf + row_b + j * 2048 + 16 * ((4 * ks + q) ^ (i16 & 7)));
    };
    constexpr int kPer = 2, kTurn = 2 * TM - 3;
    static_assert((kTurn + 3) * kPer >= LA + LB, "every load of a step has a row");
    auto step = [&](int s, auto more, auto next) {
        const uint8_t* cur = lds + (s & 1) * kStage;
        uint8_t* nxt = lds + ((s + 1) & 1) * kStage;
#pragma unroll
        for (int e = 0; e < 2 * TM; ++e) {
            if constexpr (next.value)  // what is left of the loads that the step before began
#pragma unroll
                for (int x = (e + 3) * kPer; x < (e + 4) * kPer && x < LA + LB; ++x) load_one(x);
            if (e + 3 < 2 * TM) read_a(e + 3, cur);
            if (e < TM)
#pragma unroll
                for (int j = e * TN / TM; j < (e + 1) * TN / TM; ++j) read_b(1, j, cur);
            if constexpr (next.value) {
                if (e == kTurn) {
                    __syncthreads();
                    if constexpr (more.value) load_begin(s + 2, lds + (s & 1) * kStage);
                }
                if (e >= kTurn) {
                    const int x = e - kTurn;
                    if constexpr (more.value)
#pragma unroll
                        for (int y = x * kPer; y < (x + 1) * kPer; ++y) load_one(y);
#pragma unroll
                    for (int j = x * TN / 3; j < (x + 1) * TN / 3; ++j) read_b(0, j, nxt);
                    read_a(x, nxt);
                }
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) mfma(acc[e % TM][j], fa[e & 3], fb[e / TM][j]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    if (total > 0) {
        load_begin(0, lds);
#pragma unroll
        for (int x = 0; x < LA + LB; ++x) load_one(x);
        __syncthreads();
        if (total > 1) {
            load_begin(1, lds + kStage);
#pragma unroll
            for (int x = 0; x < 3 * kPer; ++x) load_one(x);
        }
#pragma unroll
        for (int j = 0; j < TN; ++j) read_b(0, j, lds);
#pragma unroll
        for (int x = 0; x < 3; ++x) read_a(x, lds);
        int s = 0;
        for (; s + 2 < total; ++s) step(s, yes, yes);
        if (s + 1 < total) step(s++, no, yes);
        step(s, no, no);
    }
    settle(acc);
}

// Where a lane's values lie: acc[t][j][r] is m = mb + m_of(t) + r, n = nb + j.
template <class T, int S>
struct Lane {
    static __device__ __forceinline__ constexpr int m_of(int t) { return 16 * S * (t / S) + 4 * (t % S); }
    int lane, wave, q, i16, mw, mb, nw, nb;
    __device__ __forceinline__ Lane(int m0, int n0) {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        q = lane >> 4;
        i16 = lane & 15;
        mw = m0 + wave / T::WN * T::TM * 16;
        mb = mw + 4 * S * q;
        nw = n0 + wave % T::WN * T::TN * 16;
        nb = nw + T::TN * i16;
    }
};

template <class T, int RUNS>
__global__ __launch_bounds__(256, T::TM > 4 ? 1 : 2) void logits_fwd(VocabGemm p) {
    constexpr int TM = T::TM, TN = T::TN;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[T::kLds];
    const int n_rows = min(p.n, *p.count);
    const Place place = {(p.m + T::BM - 1) / T::BM, (n_rows + T::BN - 1) / T::BN};
    const int id = tile_of(blockIdx.x, place.mt * place.nt);
    if (id < 0) return;
    int m0, n0;
    place.of(id, &m0, &n0);
    m0 *= T::BM;
    n0 *= T::BN;
    f32x4 acc[TM][TN];
    product<T, RUNS, 1>(p, m0, n0, n_rows, 0, p.k / kVocabStep, lds, acc);
    const Lane<T, 1> l(m0, n0);

    // a row's largest logit and sum of exponentials over the wave's vocabulary
    float top[TN], sum[TN];
    auto statistics = [&](auto whole) {
        auto there = [&](int t, int r) { return whole.value || l.mb + l.m_of(t) + r < p.m; };
        auto largest = [&](auto up) {
            const float sign = up.value ? 1.0f : -1.0f;
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                float m = -__builtin_inff();
#pragma unroll
                for (int t = 0; t < TM; ++t) {
                    const f32x4 v = take(acc[t][j]);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (there(t, r)) m = fmaxf(m, sign * v[r]);
                }
                top[j] = m * (sign * p.scale2);
            }
        };
        if (p.scale2 >= 0.0f) largest(yes);
        else largest(no);
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            float m = fmaxf(top[j], __shfl_xor(top[j], 16));
            m = fmaxf(m, __shfl_xor(m, 32));
            // nothing is taken off an infinite maximum: all -inf sum to 0, +inf to +inf
            const bool none = !(m > -__builtin_inff());
            m = fabsf(m) < __builtin_inff() ? m : 0.0f;
            float s = 0.0f;
#pragma unroll
            for (int t = 0; t < TM; ++t) {
                const f32x4 v = take(acc[t][j]);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (there(t, r)) s += fast_exp2(fmaf(v[r], p.scale2, -m));
            }
            s += __shfl_xor(s, 16);
            s += __shfl_xor(s, 32);
            top[j] = none ? -0x1p127f : m;  // a sum of nothing, under every other
            sum[j] = s;
        }
    };
    if (l.mw + TM * 16 <= p.m) statistics(yes);
    else statistics(no);
    if (l.q == 0) {
        float4* to = reinterpret_cast<float4*>(p.part + (int64_t)(l.mw / (TM * 16)) * p.Np + l.nb);
#pragma unroll
        for (int j = 0; j < TN; j += 2) to[j / 2] = make_float4(top[j], sum[j], top[j + 1], sum[j + 1]);
    }

    // The logits at the rows' ids, 64 ids a row at a time: which of a lane's rows' ids
    // are in the wave's vocabulary, as bits, then 64 of m at a time through LDS.
    constexpr int U = TM / 4, X = TN / 4, kIds = 16;
    const int base = p.v0 + l.mw, left = max(min(p.m - l.mw, 16 * TM), 0);
    uint32_t window[X];  // of the vocabulary, for the lane's rows
#pragma unroll
    for (int x = 0; x < X; ++x) window[x] = l.nw + 64 * x + l.lane < n_rows ? left : 0;
    float* mine = reinterpret_cast<float*>(lds + l.wave * (TN * 4096));
    __syncthreads();
    for (int k0 = 0; k0 < p.K; k0 += 64) {
        // `ats` holds where a row's last ten are, 6 bits each
        uint64_t hits[U][X] = {}, ats[U][X] = {};
        const int some = min(64, p.K - k0);
        for (int k1 = 0; k1 < some; k1 += kIds) {
            int id[kIds][X];
#pragma unroll
            for (int k = 0; k < kIds; ++k)
#pragma unroll
                for (int x = 0; x < X; ++x)
                    if (k1 + k < some)
                        id[k][x] = p.kid[(k0 + k1 + k) * p.Np + min(l.nw + 64 * x + l.lane, n_rows - 1)];
#pragma unroll
            for (int k = 0; k < kIds; ++k)
                if (k1 + k < some)
#pragma unroll
                    for (int x = 0; x < X; ++x) {
                        // an absent entry's id is -1
                        const uint32_t at = id[k][x] - base;
                        if (at < window[x]) {
#pragma unroll
                            for (int u = 0; u < U; ++u)
                                if (at / 64 == u) {
                                    hits[u][x] |= 1ull << (k1 + k);
                                    ats[u][x] = ats[u][x] << 6 | (at & 63);
                                }
                        }
                    }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            bool any = false;
#pragma unroll
            for (int x = 0; x < X; ++x) any |= hits[u][x] != 0;
            if (!__any(any)) continue;
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    *reinterpret_cast<f32x4*>(mine + (TN * l.i16 + j) * 64 + 4 * ((4 * s + l.q) ^ l.i16)) =
                        take(acc[4 * u + s][j]);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int x = 0; x < X; ++x)
                for (int y = 0; hits[u][x]; ++y) {
                    const int k = 63 - __builtin_clzll(hits[u][x]), n = 64 * x + l.lane;
                    hits[u][x] &= ~(1ull << k);
                    const int64_t e = (int64_t)(k0 + k) * p.Np + l.nw + n;
                    const int at = y < 10 ? (int)(ats[u][x] & 63) : p.kid[e] - base - 64 * u;
                    ats[u][x] >>= 6;
                    p.slog[e] = p.scale2 * mine[n * 64 + 4 * ((at >> 2) ^ (n / TN)) + (at & 3)];
                }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
    }
}

// GT: g's terms
template <class T, int RUNS, int GT>
__global__ __launch_bounds__(256, T::TM > 4 ? 1 : 2) void logits_bwd(VocabGemm p) {
    constexpr int TM = T::TM, TN = T::TN;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[T::kLds];
    const int n_rows = min(p.n, *p.count);
    const Place place = {(p.m + T::BM - 1) / T::BM, (n_rows + T::BN - 1) / T::BN};
    const int id = tile_of(blockIdx.x, place.mt * place.nt);
    if (id < 0) return;
    int m0, n0;
    place.of(id, &m0, &n0);
    m0 *= T::BM;
    n0 *= T::BN;
    f32x4 acc[TM][TN];
    product<T, RUNS, 2>(p, m0, n0, n_rows, 0, p.k / kVocabStep, lds, acc);
    const Lane<T, 2> l(m0, n0);

    float lse2[TN], coef[TN];
    __builtin_memcpy(lse2, p.lse2 + l.nb, sizeof lse2);
    __builtin_memcpy(coef, p.coef + l.nb, sizeof coef);
    const int64_t plane = p.Np * p.ld_g;
    // two tiles, 8 neighbouring m, at a time; zero past the vocabulary and the rows
    auto store = [&](int t0, auto whole) {
        float v[2][TN][4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const f32x4 c = take(acc[t0 + t][j]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool there = whole.value || (l.nb + j < n_rows && l.mb + l.m_of(t0 + t) + r < p.m);
                    const float x = coef[j] * fast_exp2(fmaf(c[r], p.scale2, -lse2[j]));
                    v[t][j][r] = there ? x : 0.0f;
                }
            }
        const int m = l.mb + l.m_of(t0);
#pragma unroll
        for (int n = 0; n < GT; ++n) {
            uint16_t g[2][TN][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) g[t][j][r] = next_term<GT>(v[t][j][r]);
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                u32x4 w;
#pragma unroll
                for (int x = 0; x < 4; ++x) w[x] = g[x / 2][j][x % 2 * 2] | (uint32_t)g[x / 2][j][x % 2 * 2 + 1] << 16;
                stream_out(p.g + n * plane + (int64_t)(l.nb + j) * p.ld_g + m, w);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    uint32_t w[TN / 2];
#pragma unroll
                    for (int j = 0; j < TN; j += 2) w[j / 2] = g[t][j][r] | (uint32_t)g[t][j + 1][r] << 16;
                    stream_out(p.gt + n * plane + (int64_t)(m + 4 * t + r) * p.Np + l.nb, w);
                }
        }
    };
    const bool whole = l.mw + TM * 16 <= p.m && l.nw + TN * 16 <= n_rows;
#pragma unroll
    for (int t = 0; t < TM; t += 2)
        if (whole) store(t, yes);
        else store(t, no);
}

template <class T, int RUNS>
__device__ __forceinline__ void tile_d_h(const VocabGemm& p, int n_rows, const Place& place, int parts, int id,
                                         uint8_t* lds) {
    constexpr int TM = T::TM, TN = T::TN;
    int m0, n0;
    const int tiles = place.mt * place.nt, split = id / tiles, all = p.k / kVocabStep;
    place.of(id - split * tiles, &m0, &n0);
    f32x4 acc[TM][TN];
    product<T, RUNS, 1>(p, m0 *= T::BM, n0 *= T::BN, n_rows, (int)((int64_t)all * split / parts),
                        (int)((int64_t)all * (split + 1) / parts), lds, acc);
    const Lane<T, 1> l(m0, n0);
    float* out = static_cast<float*>(p.out) + (int64_t)split * place.nt * T::BN * p.ld_out;
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int t = 0; t < TM; ++t) {
            const int m = l.mb + l.m_of(t);
            if (l.nb + j >= n_rows || m >= p.ld_out) continue;  // ld_out: m's padded end
            f32x4* to = reinterpret_cast<f32x4*>(out + (int64_t)(l.nb + j) * p.ld_out + m);
            const f32x4 v = take(acc[t][j]);
            stream_out(to, p.accumulate ? *to + v : v);
        }
}

template <class T, int RUNS>
__device__ __forceinline__ void tile_d_w(const VocabGemm& p, int count, const Place& place, int id, uint8_t* lds) {
    constexpr int TM = T::TM, TN = T::TN, S = RUNS == 6 ? 1 : 2;
    int m0, n0;
    const int tiles = place.mt * place.nt, split = id / tiles, all = (count + kVocabStep - 1) / kVocabStep;
    place.of(id - split * tiles, &m0, &n0);
    f32x4 acc[TM][TN];
    product<T, RUNS, S>(p, m0 *= T::BM, n0 *= T::BN, p.n, (int)((int64_t)all * split / p.splits),
                        (int)((int64_t)all * (split + 1) / p.splits), lds, acc);
    const Lane<T, S> l(m0, n0);
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int t = 0; t < TM; t += S) {
            const int m = l.mb + l.m_of(t), left = p.m - m;
            if (l.nb + j >= p.n || left <= 0) continue;
            float v[4 * S];
#pragma unroll
            for (int x = 0; x < S; ++x) {
                const f32x4 c = take(acc[t + x][j]);
#pragma unroll
                for (int r = 0; r < 4; ++r) v[4 * x + r] = c[r];
            }
            const int64_t at = split * p.out_part + (int64_t)(l.nb + j) * p.ld_out + m;
            if (p.out_dtype == SSM_F32) store_dw(static_cast<float*>(p.out) + at, v, left, p.accumulate);
            else store_dw(static_cast<bf16_t*>(p.out) + at, v, left, p.accumulate);
        }
}

// Both products in one launch, so that the compute units that one's last round of
// tiles leaves idle take the other's.
template <class T, int RUNS>
__global__ __launch_bounds__(256, T::TM > 4 ? 1 : 2) void grads(VocabGemm h, VocabGemm w) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[T::kLds];
    const int count = *h.count, n_h = min(h.n, count);
    const Place ph = {(h.m + T::BM - 1) / T::BM, (n_h + T::BN - 1) / T::BN};
    const Place pw = {(w.m + T::BM - 1) / T::BM, (w.n + T::BN - 1) / T::BN};
    // every XCD takes its part of d_h, whose sums are longer as a rule, then of d_w
    const int parts = h.split.of(ph.nt);
    const int tiles_h = ph.mt * ph.nt * parts, pid = blockIdx.x, first = (int)on_xcds(tiles_h);
    if (pid < first) {
        const int id = tile_of(pid, tiles_h);
        if (id >= 0) tile_d_h<T, RUNS>(h, n_h, ph, parts, id, lds);
    } else {
        const int id = tile_of(pid - first, pw.mt * pw.nt * w.splits);
        if (id >= 0) tile_d_w<T, RUNS>(w, count, pw, id, lds);
    }
}

// Whether 256 x 256 tiles, one a compute unit, take less time than 128 x 128 tiles, two a
// compute unit.  A round of tiles takes `steps` steps of k, 1.48 us each (a big tile's)
// or 0.88, and its results: `big` or `small` us, measured with sums of 5 and of 40
// steps.  (16384 x 32768 logits: width 2560 1946 us in big tiles, 2313 in small ones;
// width 320 440 and 423 us.)
struct Results {
    double big, small;
};
constexpr Results kStatistics = {5.0, 2.0}, kBothOrders = {13.0, 8.0};

bool big_tiles(int64_t big, int64_t small, double steps, Results r) {
    return ((big + 255) / 256) * (1.48 * steps + r.big) <= ((small + 511) / 512) * (0.88 * steps + r.small);
}

bool big_logits(const VocabGemm& g, int terms, Results r) {
    const double steps = (terms == 3 ? 6 : 1) * (g.k / kVocabStep);
    return big_tiles(vocab_tiles(g.m, g.n, 256), vocab_tiles(g.m, g.n, 128), steps, {r.big * terms, r.small * terms});
}

int launched() { return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP; }

template <class T>
int launch_fwd(const VocabGemm& g, int terms, hipStream_t stream) {
    const unsigned grid = (unsigned)on_xcds(vocab_tiles(g.m, g.n, T::BM));
    if (terms == 1) logits_fwd<T, 1><<<grid, 256, 0, stream>>>(g);
    else logits_fwd<T, 6><<<grid, 256, 0, stream>>>(g);
    return launched();
}

template <class T>
int launch_bwd(const VocabGemm& g, int terms, hipStream_t stream) {
    const unsigned grid = (unsigned)on_xcds(vocab_tiles(g.m, g.n, T::BM));
    if (terms == 3) logits_bwd<T, 6, 3><<<grid, 256, 0, stream>>>(g);
    else logits_bwd<T, 1, 1><<<grid, 256, 0, stream>>>(g);
    return launched();
}

template <class T>
unsigned grads_grid(const VocabGemm& h, const VocabGemm& w) {
    return (unsigned)on_xcds(vocab_tiles(h.m, h.n, T::BM) * h.split.parts) + (unsigned)on_xcds(vocab_tiles(w.m, w.n, T::BM) * w.splits);
}

template <class T>
int launch_grads(const VocabGemm& h, const VocabGemm& w, int terms, hipStream_t stream) {
    if (terms == 3) grads<T, 6><<<grads_grid<T>(h, w), 256, 0, stream>>>(h, w);
    else grads<T, 1><<<grads_grid<T>(h, w), 256, 0, stream>>>(h, w);
    return launched();
}

}  // namespace

int vocab_parts(const VocabGemm& g, int terms) {
    return big_logits(g, terms, kStatistics) ? (g.m + 255) / 256 * 2 : (g.m + 127) / 128 * 2;
}

int launch_vocab_logits_fwd(const VocabGemm& g, int terms, hipStream_t stream) {
    return big_logits(g, terms, kStatistics) ? launch_fwd<Big>(g, terms, stream) : launch_fwd<Small>(g, terms, stream);
}

int launch_vocab_logits_bwd(const VocabGemm& g, int terms, hipStream_t stream) {
    return big_logits(g, terms, kBothOrders) ? launch_bwd<Big>(g, terms, stream) : launch_bwd<Small>(g, terms, stream);
}

int launch_vocab_grads(const VocabGemm& h, const VocabGemm& w, int terms, bool big, hipStream_t stream) {
    return big ? launch_grads<Big>(h, w, terms, stream) : launch_grads<Small>(h, w, terms, stream);
}

}  // namespace ssm
