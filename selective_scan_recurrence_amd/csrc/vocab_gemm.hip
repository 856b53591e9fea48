// The products of the losses over a vocabulary: out[n][m] = sum_k A[m][k] B[n][k],
// both operands with k fastest, in bf16 on MFMA with f32 sums.
//   logits:  A = W (m: vocabulary), B = h (n: rows);  forward: the softmax
//            statistics of each row over the tile's vocabulary, and the logits at
//            the row's ids; backward: g = coef exp2(s - lse), stored in both
//            orders, since one product sums over the vocabulary and one over rows
//   d_h:     A = W turned (m: width),  B = g (n: rows)
//   d_W:     A = h turned (m: width),  B = g turned (n: vocabulary)
// An f32 value is three bf16 terms, and a product the six of its nine partial
// products that reach 2^-24 of it, the small ones first: six runs over k.
//
// A workgroup owns BM x BN of out and walks k in steps of 64: 128-byte rows go
// from memory to LDS past the registers, into one of two buffers while the
// other is multiplied.  A row's 16-byte piece c sits at c ^ f(row).  MFMA tile t of a
// wave's rows takes rows 64 (t / 4) + 16 (i / 4) + 4 (t % 4) + i % 4 (i = 0 ..
// 15), and tile j of its 64 columns the columns 4 i + j: a lane (q = lane / 16,
// i = lane % 16) then holds 16 neighbouring m (from 16 q) and 4 neighbouring n
// (from 4 i), so that both orders leave in 8- to 16-byte stores.  With f = i % 8 for
// both, any 8 neighbouring lanes of a read meet 8 different pieces.
#include "vocab.h"

namespace ssm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void* lds_ptr;

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

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return (uint32_t)bf16_rne(lo) | (uint32_t)bf16_rne(hi) << 16;
}

// planes of the six partial products, small ones first
__device__ __forceinline__ int plane_a(int t) { return (0x001102 >> (4 * t)) & 15; }
__device__ __forceinline__ int plane_b(int t) { return (0x010120 >> (4 * t)) & 15; }

template <int WM, int WN, int TM, int MODE, int TERMS>
__global__ __launch_bounds__(64 * WM * WN, WM * WN >= 8 ? 2 : 2) void vocab_gemm(VocabGemm p) {
    constexpr int NW = WM * WN, BM = WM * TM * 16, BN = WN * 64, U = TM / 4;
    constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;
    constexpr int kStage = (BM + BN) * 128;
    static_assert(2 * kStage >= NW * 16384, "the logits at the ids pass through LDS");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kStage];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN, q = lane >> 4, i16 = lane & 15;

    const int count = p.count ? *p.count : 0;
    const int n_rows = MODE == kGradW ? p.n : min(p.n, count);
    const int k_len = MODE == kGradW ? (count + kVocabStep - 1) / kVocabStep * kVocabStep : p.k;
    const int mt = (p.m + BM - 1) / BM, nt = (n_rows + BN - 1) / BN, total = mt * nt;
    // workgroups are dealt to the 8 XCDs in turn: an XCD's are neighbouring
    // tiles, 8 columns of tiles wide, that share A and B
    const int split = blockIdx.y;
    const int per = (total + 7) / 8, pid = blockIdx.x;
    const int id = pid % 8 * per + pid / 8;
    if (pid / 8 >= per || id >= total) return;
    const int band = id / (mt * 8), in = id - band * mt * 8, wide = min(8, nt - 8 * band);
    const int m0 = in / wide * BM, n0 = (8 * band + in % wide) * BN;

    // k of this split, in steps
    int s_begin = 0, s_end = k_len / kVocabStep;
    if (p.splits > 1) {
        const int all = s_end;
        s_begin = (int)((int64_t)all * split / p.splits);
        s_end = (int)((int64_t)all * (split + 1) / p.splits);
    }
    const int steps = s_end - s_begin, total_steps = TERMS == 1 ? steps : 6 * steps;

    // loads: a wave's load is 8 rows of 8 pieces
    uint32_t at_a[LA], at_b[LB];
#pragma unroll
    for (int x = 0; x < LA; ++x) {
        const int row = 8 * (wave + NW * x) + lane / 8, f = (row & 3) | (row >> 4 & 1) << 2;
        at_a[x] = (uint32_t)min(row, p.m - 1 - m0) * (uint32_t)(2 * p.lda) + 16 * ((lane & 7) ^ f);
    }
#pragma unroll
    for (int x = 0; x < LB; ++x) {
        const int row = 8 * (wave + NW * x) + lane / 8, f = row >> 2 & 7;
        at_b[x] = (uint32_t)min(row, n_rows - 1 - n0) * (uint32_t)(2 * p.ldb) + 16 * ((lane & 7) ^ f);
    }
    const uint16_t* a = p.a + (int64_t)m0 * p.lda + (int64_t)s_begin * kVocabStep;
    const uint16_t* b = p.b + (int64_t)n0 * p.ldb + (int64_t)s_begin * kVocabStep;
    auto load = [&](int step, uint8_t* buf) {
        const int term = TERMS == 1 ? 0 : step / steps, s = TERMS == 1 ? step : step - term * steps;
        const auto ra = rsrc_of(TERMS == 1 ? a : a + plane_a(term) * p.a_plane);
        const auto rb = rsrc_of(TERMS == 1 ? b : b + plane_b(term) * p.b_plane);
#pragma unroll
        for (int x = 0; x < LA; ++x) load_lds(ra, buf + (wave + NW * x) * 1024, at_a[x], s * (2 * kVocabStep));
#pragma unroll
        for (int x = 0; x < LB; ++x)
            load_lds(rb, buf + BM * 128 + (wave + NW * x) * 1024, at_b[x], s * (2 * kVocabStep));
    };

    f32x4 acc[TM][4];
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t][j] = f32x4{0, 0, 0, 0};
    const uint32_t row_a = (wm * TM * 16 + 16 * (i16 >> 2) + (i16 & 3)) * 128;
    const uint32_t row_b = BM * 128 + (wn * 64 + 4 * i16) * 128;
    auto multiply = [&](const uint8_t* buf) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const uint32_t c = 16 * ((4 * ks + q) ^ (i16 & 7));
            u32x4 fa[TM], fb[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) fb[j] = *reinterpret_cast<const u32x4*>(buf + row_b + j * 128 + c);
#pragma unroll
            for (int t = 0; t < TM; ++t)
                fa[t] = *reinterpret_cast<const u32x4*>(buf + row_a + (64 * (t / 4) + 4 * (t % 4)) * 128 + c);
#pragma unroll
            for (int t = 0; t < TM; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[t][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, fa[t]), __builtin_bit_cast(bf16x8, fb[j]), acc[t][j], 0, 0, 0);
        }
    };
    if (total_steps > 0) load(0, lds);
    for (int s = 0; s < total_steps; ++s) {
        __syncthreads();
        if (s + 1 < total_steps) load(s + 1, lds + (s + 1 & 1) * kStage);
        multiply(lds + (s & 1) * kStage);
    }

    // lane (q, i): acc[4 u + s][j][r] is m = mb + 64 u + 4 s + r, n = nb + j
    const int mw = m0 + wm * TM * 16, mb = mw + 16 * q, nw = n0 + wn * 64, nb = nw + 4 * i16;
    if constexpr (MODE == kLogitsFwd) {
        float top[4], sum[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float m = -__builtin_inff();
#pragma unroll
            for (int t = 0; t < TM; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool there = mb + 64 * (t / 4) + 4 * (t % 4) + r < p.m;
                    const float v = there ? acc[t][j][r] * p.scale2 : -__builtin_inff();
                    acc[t][j][r] = v;
                    m = fmaxf(m, v);
                }
            m = fmaxf(m, __shfl_xor(m, 16));
            m = fmaxf(m, __shfl_xor(m, 32));
            // nothing is taken off an infinite maximum: all -inf sum to 0, +inf to +inf
            const bool none = m == -__builtin_inff();
            m = fabsf(m) < __builtin_inff() ? m : 0.0f;
            float l = 0.0f;
#pragma unroll
            for (int t = 0; t < TM; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) l += fast_exp2(acc[t][j][r] - m);
            l += __shfl_xor(l, 16);
            l += __shfl_xor(l, 32);
            top[j] = none ? -0x1p127f : m;  // a sum of nothing, under every other
            sum[j] = l;
        }
        if (q == 0) {
            float4* to = reinterpret_cast<float4*>(p.part + (int64_t)(m0 / (TM * 16) + wm) * p.Np + nb);
            to[0] = make_float4(top[0], sum[0], top[1], sum[1]);
            to[1] = make_float4(top[2], sum[2], top[3], sum[3]);
        }
        // the logits at the rows' ids: 64 of m at a time through LDS, a token a lane
        __syncthreads();
        float* mine = reinterpret_cast<float*>(lds + wave * 16384);
        const int n = nw + lane;
        const int32_t* ids = p.kid + (int64_t)min(n, n_rows - 1) * p.K;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int base = p.v0 + mw + 64 * u, top_m = min(64, p.m - mw - 64 * u);
            bool any = false;
            for (int k = 0; k < p.K; ++k) any |= ids[k] >= base && ids[k] - base < top_m;
            if (!__any(any && n < n_rows)) continue;
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<f32x4*>(mine + (4 * i16 + j) * 64 + 4 * ((4 * q + s) ^ i16)) = acc[4 * u + s][j];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (n < n_rows)
                for (int k = 0; k < p.K; ++k) {
                    const int at = ids[k] - base;
                    if (ids[k] >= base && at < top_m)
                        p.slog[(int64_t)n * p.K + k] = mine[lane * 64 + 4 * ((at >> 2) ^ (lane >> 2)) + (at & 3)];
                }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
    } else if constexpr (MODE == kLogitsBwd) {
        const float4 l4 = *reinterpret_cast<const float4*>(p.lse2 + nb), c4 = *reinterpret_cast<const float4*>(p.coef + nb);
        const float lse2[4] = {l4.x, l4.y, l4.z, l4.w}, coef[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int t = 0; t < TM; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool there = nb + j < n_rows && mb + 64 * (t / 4) + 4 * (t % 4) + r < p.m;
                    acc[t][j][r] = there ? coef[j] * fast_exp2(fmaf(acc[t][j][r], p.scale2, -lse2[j])) : 0.0f;
                }
#pragma unroll
        for (int term = 0; term < TERMS; ++term) {
            // this term of every value, and what it leaves for the next
            uint32_t half[TM][4][2];
#pragma unroll
            for (int t = 0; t < TM; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (TERMS == 1) {
                        half[t][j][0] = pack2(acc[t][j][0], acc[t][j][1]);
                        half[t][j][1] = pack2(acc[t][j][2], acc[t][j][3]);
                    } else {
                        uint32_t w[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float v = acc[t][j][r];
                            w[r] = v != v ? 0x7fc0u : __float_as_uint(v) >> 16;
                            acc[t][j][r] = fabsf(v) < __builtin_inff() ? v - __uint_as_float(w[r] << 16) : 0.0f;
                        }
                        half[t][j][0] = w[0] | w[1] << 16;
                        half[t][j][1] = w[2] | w[3] << 16;
                    }
                }
            uint16_t* g = p.g + term * (p.Np * p.P);
            uint16_t* gt = p.gt + term * (p.Np * p.P);
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int t = 4 * u + 2 * h;
                        *reinterpret_cast<u32x4*>(g + (int64_t)(nb + j) * p.P + mb + 64 * u + 8 * h) =
                            u32x4{half[t][j][0], half[t][j][1], half[t + 1][j][0], half[t + 1][j][1]};
                    }
#pragma unroll
            for (int t = 0; t < TM; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint32_t sel = r & 1 ? 0x07060302u : 0x05040100u;
                    const u32x2 v = {__builtin_amdgcn_perm(half[t][1][r / 2], half[t][0][r / 2], sel),
                                     __builtin_amdgcn_perm(half[t][3][r / 2], half[t][2][r / 2], sel)};
                    const int m = mb + 64 * (t / 4) + 4 * (t % 4) + r;
                    *reinterpret_cast<u32x2*>(gt + (int64_t)m * p.Np + nb) = v;
                }
        }
    } else if constexpr (MODE == kGradH) {
        float* out = static_cast<float*>(p.out) + split * p.split_stride;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int t = 0; t < TM; ++t) {
                const int m = mb + 64 * (t / 4) + 4 * (t % 4);
                if (nb + j >= n_rows || m >= p.ld_out) continue;  // ld_out: m's padded end
                f32x4* to = reinterpret_cast<f32x4*>(out + (int64_t)(nb + j) * p.ld_out + m);
                *to = p.accumulate ? *to + acc[t][j] : acc[t][j];
            }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int t = 0; t < TM; ++t) {
                const int m = mb + 64 * (t / 4) + 4 * (t % 4), left = p.m - m;
                if (nb + j >= n_rows || left <= 0) continue;
                const int64_t at = (int64_t)(nb + j) * p.ld_out + m;
                f32x4 v = acc[t][j];
                if (p.out_dtype == SSM_F32) {
                    float* to = static_cast<float*>(p.out) + at;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (p.accumulate && r < left) v[r] += to[r];
                    if (left >= 4) __builtin_memcpy(to, &v, 16);
                    else
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (r < left) to[r] = v[r];
                } else {
                    uint16_t* to = static_cast<uint16_t*>(p.out) + at;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (p.accumulate && r < left) v[r] += to_f32(to[r]);
                    const u32x2 w = {pack2(v[0], v[1]), pack2(v[2], v[3])};
                    if (left >= 4) __builtin_memcpy(to, &w, 8);
                    else
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (r < left) to[r] = bf16_rne(v[r]);
                }
            }
    }
}

template <int WM, int WN, int TM, int MODE>
int launch(const VocabGemm& g, hipStream_t stream) {
    constexpr int BM = WM * TM * 16, BN = WN * 64;
    const int64_t mt = (g.m + BM - 1) / BM, nt = (g.n + BN - 1) / BN, total = (mt * nt + 7) / 8 * 8;
    const dim3 grid((unsigned)total, (unsigned)g.splits);
    if (g.terms == 1) vocab_gemm<WM, WN, TM, MODE, 1><<<grid, 64 * WM * WN, 0, stream>>>(g);
    else vocab_gemm<WM, WN, TM, MODE, 3><<<grid, 64 * WM * WN, 0, stream>>>(g);
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

template <int MODE>
int launch_mode(const VocabGemm& g, hipStream_t stream) {
    return launch<2, 2, 4, MODE>(g, stream);
}

}  // namespace

int vocab_parts(int m, int) { return (m + 127) / 128 * 2; }

int launch_vocab_gemm(const VocabGemm& g, hipStream_t stream) {
    if (g.m <= 0 || g.n <= 0) return SSM_OK;
    switch (g.mode) {
        case kLogitsFwd: return launch_mode<kLogitsFwd>(g, stream);
        case kLogitsBwd: return launch_mode<kLogitsBwd>(g, stream);
        case kGradH: return launch_mode<kGradH>(g, stream);
        default: return launch_mode<kGradW>(g, stream);
    }
}

}  // namespace ssm
