// The losses over a vocabulary, around their products: which rows count, the
// operands' layouts, the join of the softmax statistics, the gradient at the
// ids, and d_h's rows.  All bound by memory or by launches; together a few
// percent of the products' time.
#include "vocab.h"

namespace ssm {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float fast_log2(float v) { return __builtin_amdgcn_logf(v); }

// A teacher's entry that counts: its id is no padding and it has some mass.
__device__ __forceinline__ bool present(const VocabRows& r, int64_t e) {
    return r.id[e] >= 0 && !(r.logit && r.logit[e] == -__builtin_inff());
}

__device__ __forceinline__ int row_state(const VocabRows& r, int i) {
    int state = kRowOut;
    for (int k = 0; k < r.K; ++k) {
        const int64_t e = (int64_t)i * r.K + k;
        if (!present(r, e)) continue;
        if (r.id[e] >= r.V) return kRowBad;
        state = 0;
    }
    return state;
}

// the same by a group of LANES neighbouring lanes
template <int LANES>
__device__ __forceinline__ int row_state_by(const VocabRows& r, int i, int lane) {
    int best = 0;  // 1: an entry that counts, 2: one past the vocabulary
    for (int k = lane; k < r.K; k += LANES) {
        const int64_t e = (int64_t)i * r.K + k;
        if (present(r, e)) best = max(best, r.id[e] >= r.V ? 2 : 1);
    }
#pragma unroll
    for (int d = 1; d < LANES; d *= 2) best = max(best, __shfl_xor(best, d));
    return best == 0 ? kRowOut : best == 1 ? 0 : kRowBad;
}

__global__ __launch_bounds__(256) void rows_state(VocabRows r, uint32_t* err) {
    const int i = blockIdx.x * 16 + threadIdx.x / 16, lane = threadIdx.x & 15;
    if (i >= r.N) return;
    const int state = row_state_by<16>(r, i, lane);
    if (lane) return;
    r.pos[i] = state;
    if (state == kRowBad && err) atomicOr(err, (uint32_t)SSM_DEVERR_TARGET);
}

// The rows that count, in order, by one workgroup, 1024 X in a round.  With one entry a
// row (a target) the states are found here.
template <int X>
__global__ __launch_bounds__(1024) void rows_list(VocabRows r, uint32_t* err) {
    __shared__ int before[X * 16], total;  // rows that count before a 64 of them (x, wave), and in all
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int done = 0;
    for (int64_t base = 0; base < r.N; base += 1024 * X) {
        int state[X];
#pragma unroll
        for (int x = 0; x < X; ++x) {
            const int i = (int)min(base + 1024 * x + tid, (int64_t)r.N - 1);
            state[x] = r.K > 1 ? r.pos[i] : row_state(r, i);
        }
        uint64_t mask[X];
#pragma unroll
        for (int x = 0; x < X; ++x) {
            if (base + 1024 * x + tid >= r.N) state[x] = kRowOut;
            if (r.K == 1 && state[x] == kRowBad && err) atomicOr(err, (uint32_t)SSM_DEVERR_TARGET);
            mask[x] = __ballot(state[x] >= 0);
            if (lane == 0) before[x * 16 + wave] = __popcll(mask[x]);
        }
        __syncthreads();
        if (wave == 0) {
            constexpr int Y = X / 4;  // of `before` a lane
            int v[Y], sum = 0;
#pragma unroll
            for (int y = 0; y < Y; ++y) {
                v[y] = sum;
                sum += before[lane * Y + y];
            }
            int up = sum;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const int w = __shfl_up(up, d);
                if (lane >= d) up += w;
            }
#pragma unroll
            for (int y = 0; y < Y; ++y) before[lane * Y + y] = done + up - sum + v[y];
            if (lane == 63) total = done + up;
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < X; ++x) {
            const int64_t i = base + 1024 * x + tid;
            if (i >= r.N) break;
            const int c = before[x * 16 + wave] + __popcll(mask[x] & ((1ull << lane) - 1));
            r.pos[i] = state[x] >= 0 ? c : state[x];
            if (state[x] < 0) continue;
            r.rows[c] = (int)i;
            if (r.K == 1) r.kid[c] = r.id[i];
        }
        done = total;
        __syncthreads();
    }
    if (tid == 0) *r.count = done;
}

__global__ __launch_bounds__(256) void rows_ids(VocabRows r) {
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int c = (int)(x / r.K), k = (int)(x % r.K);
    if (c >= *r.count) return;
    const int64_t from = (int64_t)r.rows[c] * r.K + k;
    r.kid[(int64_t)k * r.Np + c] = present(r, from) ? r.id[from] : -1;
}

// ---- layouts ----------------------------------------------------------------

__device__ __forceinline__ const char* row_of(const VocabPack& p, int r) {
    const int64_t row = p.rows ? p.rows[r] : p.r0 + r;
    return static_cast<const char*>(p.src) + row * p.ld * (p.dtype == SSM_BF16 ? 2 : 4);
}

// eight values of a row from column c, as terms; zero past the width
template <int TERMS>
__device__ __forceinline__ void load8(const VocabPack& p, const char* row, int c, bool wide, uint16_t (&t)[TERMS][8]) {
    if constexpr (TERMS == 1) {
        const uint16_t* s = reinterpret_cast<const uint16_t*>(row) + c;
        if (wide && c + 8 <= p.width) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(s);
            __builtin_memcpy(t[0], &v, 16);
            return;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) t[0][e] = c + e < p.width ? s[e] : 0;
    } else {
        const float* s = reinterpret_cast<const float*>(row) + c;
        float v[8];
        if (wide && c + 8 <= p.width) {
            const float4 a = reinterpret_cast<const float4*>(s)[0], b = reinterpret_cast<const float4*>(s)[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = c + e < p.width ? s[e] : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint16_t w[3];
            bf16_terms<3>(v[e], w);
#pragma unroll
            for (int n = 0; n < 3; ++n) t[n][e] = w[n];
        }
    }
}

template <int TERMS>
__device__ __forceinline__ void pack_piece(const VocabPack& p, bool wide, int64_t x) {
    const int pieces = (p.width + 63) / 64 * 8;
    const int r = (int)(x / pieces), c = 8 * (int)(x % pieces);
    if (r >= (p.count ? min(p.n, *p.count) : p.n)) return;
    uint16_t t[TERMS][8];
    load8<TERMS>(p, row_of(p, r), c, wide, t);
#pragma unroll
    for (int n = 0; n < TERMS; ++n)
        __builtin_memcpy(__builtin_assume_aligned(p.out + n * p.plane + (int64_t)r * (8 * pieces) + c, 16), t[n], 16);
}

// a tile of 64 rows x 64 columns through LDS; zero where a row is not there
template <int TERMS, typename There>
__device__ __forceinline__ void turn_tile(const VocabPack& p, int r0, int c0, int n, bool wide, There there) {
    __shared__ __attribute__((aligned(16))) uint16_t tile[64][72];
    const int tid = threadIdx.x;
    uint16_t t[2][TERMS][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = r0 + 32 * h + tid / 8, c = c0 + 8 * (tid % 8);
#pragma unroll
        for (int x = 0; x < TERMS; ++x)
#pragma unroll
            for (int e = 0; e < 8; ++e) t[h][x][e] = 0;
        if (r < n && c < p.width && there(r)) load8<TERMS>(p, row_of(p, r), c, wide, t[h]);
    }
#pragma unroll
    for (int x = 0; x < TERMS; ++x) {
        if (x) __syncthreads();
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 8; ++e) tile[8 * (tid % 8) + e][32 * h + tid / 8] = t[h][x][e];
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = 32 * h + tid / 8, r = 8 * (tid % 8);
            if (c0 + c < p.width)
                *reinterpret_cast<u32x4*>(p.out + x * p.plane + (int64_t)(c0 + c) * p.ld_rows + r0 + r) =
                    *reinterpret_cast<const u32x4*>(&tile[c][r]);
        }
    }
}

bool is_wide(const VocabPack& p) {
    const int64_t es = p.dtype == SSM_BF16 ? 2 : 4;
    return reinterpret_cast<uintptr_t>(p.src) % 16 == 0 && p.ld * es % 16 == 0;
}

// ---- the teacher's probabilities -----------------------------------------------

// Logits are taken off each other before anything multiplies them: masked ones hold the
// lowest finite value, whose products with top_scale and log2 e are infinite.
struct Teacher {
    float base;  // top_lse, or half of the logit with the most mass: of halves every difference is finite
    float off;   // log2 of the sum of the entries' masses against that one's
};

// log2 p of an entry
__device__ __forceinline__ float top2(const VocabRows& r, int64_t e, const Teacher& t) {
    if (!present(r, e)) return -__builtin_inff();
    const float x = r.logit[e];
    if (r.top_lse) return fmaf(r.top_scale, x, -t.base) * kLog2e;
    return (0.5f * x - t.base) * r.top_scale * (2.0f * kLog2e) - t.off;
}

// by the 2^x lanes of a group with the same row
__device__ __forceinline__ Teacher teacher_of(const VocabRows& r, int64_t i, int lane, int lanes) {
    if (r.top_lse) return {r.top_lse[i], 0.0f};
    const float sign = r.top_scale < 0.0f ? -1.0f : 1.0f;
    float m = -__builtin_inff(), s = 0.0f;
    for (int k = lane; k < r.K; k += lanes)
        if (present(r, i * r.K + k)) m = fmaxf(m, sign * r.logit[i * r.K + k]);
    for (int d = 1; d < lanes; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
    Teacher t = {0.5f * sign * m, 0.0f};
    for (int k = lane; k < r.K; k += lanes) s += fast_exp2(top2(r, i * r.K + k, t));
    for (int d = 1; d < lanes; d *= 2) s += __shfl_xor(s, d);
    t.off = fast_log2(s);
    return t;
}

// ---- softmax statistics ----------------------------------------------------------

// sums over the LANES lanes of a row, 8, 64 or a whole workgroup
template <int LANES, typename Combine>
__device__ __forceinline__ void combine_lanes(float& m, float& s, Combine combine) {
#pragma unroll
    for (int d = 1; d < (LANES < 64 ? LANES : 64); d *= 2) combine(m, s, __shfl_xor(m, d), __shfl_xor(s, d));
    if constexpr (LANES == 256) {
        __shared__ float2 waves[4];
        __syncthreads();
        if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = make_float2(m, s);
        __syncthreads();
        m = waves[0].x;
        s = waves[0].y;
#pragma unroll
        for (int w = 1; w < 4; ++w) combine(m, s, waves[w].x, waves[w].y);
    }
}

// Few rows have many partials each: then a wave or a workgroup takes a row.
template <int LANES>
__global__ __launch_bounds__(256) void join_rows(VocabJoin j) {
    const VocabRows& r = j.r;
    const int lane = threadIdx.x % LANES;
    const int64_t i = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
    if (i >= r.N) return;
    int c;
    if (r.pos) {
        c = r.pos[i];
    } else {
        const int state = row_state_by<(LANES < 64 ? LANES : 64)>(r, (int)i, lane & 63);
        c = state < 0 ? state : (int)i;
        if (state == kRowBad && j.err && lane == 0) atomicOr(j.err, (uint32_t)SSM_DEVERR_TARGET);
    }
    if (c < 0) {
        if (!j.last) return;
        const float v = c == kRowBad ? __builtin_nanf("") : 0.0f;
        if (lane == 0) {
            if (j.loss) j.loss[i] = v;
            if (j.lse) j.lse[i] = v;
        }
        if (j.logq)
            for (int k = lane; k < r.K; k += LANES) j.logq[i * r.K + k] = v;
        return;
    }
    // a lane without a part holds a sum of nothing
    float m = -0x1p127f, s = 0.0f;
    for (int x = lane; x < j.parts; x += 4 * LANES) {
        float2 v[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
            v[y] = j.part[(int64_t)min(x + y * LANES, j.parts - 1) * r.Np + c];
#pragma unroll
        for (int y = 0; y < 4; ++y)
            if (x + y * LANES < j.parts) merge(m, s, v[y].x, v[y].y);
    }
    combine_lanes<LANES>(m, s, merge);
    if (!j.first) merge(m, s, j.state[c].x, j.state[c].y);
    if (!j.last) {
        if (LANES == 256) __syncthreads();  // every lane has read the state
        if (lane == 0) j.state[c] = make_float2(m, s);
        return;
    }
    const float l = fast_log2(s);
    if (lane == 0 && j.lse) j.lse[i] = (m + l) * kLn2;
    if (!r.logit) {
        if (lane == 0 && j.loss) j.loss[i] = ((m - j.slog[c]) + l) * kLn2;
        return;
    }
    const Teacher t = teacher_of(r, i, lane & 63, LANES < 64 ? LANES : 64);
    float loss = 0.0f, none = 0.0f;
    for (int k = lane; k < r.K; k += LANES) {
        const int64_t e = i * r.K + k;
        const bool there = present(r, e);
        const float q = there ? (j.slog[(int64_t)k * r.Np + c] - m) - l : 0.0f, log_p = top2(r, e, t);
        if (j.logq) j.logq[e] = q * kLn2;
        // p log p is 0 at 0, where its logarithm may be infinite
        const float p = fast_exp2(log_p);
        if (p != 0.0f) loss += p * (log_p - q);
    }
    combine_lanes<LANES>(none, loss, [](float&, float& a, float, float b) { a += b; });
    if (lane == 0 && j.loss) j.loss[i] = loss * kLn2;
}

// ---- the gradient's factors ---------------------------------------------------

// of row i, which counts as row c
__device__ __forceinline__ void target_factors(const VocabCoef& f, int i, int c) {
    const float d = f.scale * f.d_loss[i], a = d + (f.d_lse ? f.scale * f.d_lse[i] : 0.0f);
    f.lse2[c] = f.lse[i] * kLog2e;
    f.coef[c] = a;
    f.at[c] = a * fast_exp2(-f.loss[i] * kLog2e) - d;
}

// by a wave
__device__ __forceinline__ void top_factors(const VocabCoef& f, int64_t i, int c, int lane) {
    const VocabRows& r = f.r;
    const float d = f.scale * f.d_loss[i];
    const Teacher t = teacher_of(r, i, lane, 64);
    float mass = 1.0f;
    if (r.top_lse) {
        mass = 0.0f;
        for (int k = lane; k < r.K; k += 64) mass += fast_exp2(top2(r, i * r.K + k, t));
        for (int x = 1; x < 64; x *= 2) mass += __shfl_xor(mass, x);
    }
    const float a = d * mass + (f.d_lse ? f.scale * f.d_lse[i] : 0.0f);
    if (lane == 0) {
        f.lse2[c] = f.lse[i] * kLog2e;
        f.coef[c] = a;
    }
    const int32_t* ids = r.id + i * r.K;
    for (int k = lane; k < r.K; k += 64) {
        if (!present(r, i * r.K + k)) continue;
        float p = 0.0f;  // of every entry with this id
        for (int x = 0; x < r.K; ++x)
            if (ids[x] == ids[k]) p += fast_exp2(top2(r, i * r.K + x, t));
        f.at[(int64_t)k * r.Np + c] = a * fast_exp2(f.logq[i * r.K + k] * kLog2e) - d * p;
    }
}

// workgroups of each kind, in this order
struct Begin {
    VocabPack pack_h, pack_w, turn_h, turn_w;
    VocabCoef coef;
    unsigned pack_h_end, pack_w_end, turn_h_end, turn_w_end;
    bool wide_h, wide_w;
};

template <int TERMS>
__global__ __launch_bounds__(256) void begin(Begin b) {
    const unsigned id = blockIdx.x;
    const int tid = threadIdx.x;
    if (id < b.pack_h_end) {
        pack_piece<TERMS>(b.pack_h, b.wide_h, (int64_t)id * 256 + tid);
    } else if (id < b.pack_w_end) {
        pack_piece<TERMS>(b.pack_w, b.wide_w, (int64_t)(id - b.pack_h_end) * 256 + tid);
    } else if (id < b.turn_w_end) {
        const bool w = id >= b.turn_h_end;
        const VocabPack& p = w ? b.turn_w : b.turn_h;
        const int x = (int)(id - (w ? b.turn_h_end : b.pack_w_end)), columns = (p.width + 63) / 64;
        const int n = p.count ? min(p.n, *p.count) : p.n, r0 = x / columns * 64;
        if (r0 < n) turn_tile<TERMS>(p, r0, x % columns * 64, n, w ? b.wide_w : b.wide_h, [](int) { return true; });
    } else if (b.coef.r.logit) {
        const int c = (int)(id - b.turn_w_end) * 4 + tid / 64;
        if (c < *b.coef.r.count) top_factors(b.coef, b.coef.r.rows[c], c, tid & 63);
    } else {
        const int c = (int)(id - b.turn_w_end) * 256 + tid;
        if (c < *b.coef.r.count) target_factors(b.coef, b.coef.r.rows[c], c);
    }
}

// The first 16 workgroups take the rows' factors, a wave a row; the next turn h, 64
// columns each; in f32 the last pack it.
template <int TERMS>
__global__ __launch_bounds__(256) void few_begin(VocabCoef f, VocabPack turned, VocabPack packed, bool wide) {
    const VocabRows& r = f.r;
    const int tid = threadIdx.x, columns = (r.D + 63) / 64, id = blockIdx.x;
    constexpr int first = kVocabFew / 4;
    const int packs = first + columns;
    if (id < first) {
        const int i = id * 4 + tid / 64;
        if (i >= r.N) return;
        const int state = row_state_by<64>(r, i, tid & 63);
        if ((tid & 63) == 0) r.pos[i] = state < 0 ? state : i;
        if (state < 0) return;
        if (r.logit) top_factors(f, i, i, tid & 63);
        else if ((tid & 63) == 0) target_factors(f, i, i);
        return;
    }
    if (id >= packs) {
        pack_piece<TERMS>(packed, wide, (int64_t)(id - packs) * 256 + tid);
        return;
    }
    __shared__ int state[kVocabFew];
    if (tid / 4 < r.N) {
        const int of = row_state_by<4>(r, tid / 4, tid & 3);
        state[tid / 4] = of;
    }
    __syncthreads();
    turn_tile<TERMS>(turned, 0, (id - first) * 64, r.N, wide, [&](int row) { return state[row] >= 0; });
}

template <int TERMS>
__global__ __launch_bounds__(256) void patch_ids(VocabPatch p, int groups) {
    const int k = blockIdx.x / groups, c = blockIdx.x % groups * 256 + threadIdx.x;
    if (c >= *p.r.count) return;
    const int64_t e = (int64_t)k * p.r.Np + c;
    const int id = p.r.kid[e], v = id - p.v0;
    if (id < p.v0 || v >= p.n) return;
    uint16_t t[TERMS];
    bf16_terms<TERMS>(p.at[e], t);
#pragma unroll
    for (int n = 0; n < TERMS; ++n)
        p.g[n * p.plane + (int64_t)c * p.ld_g + v] = p.gt[n * p.plane + (int64_t)v * p.r.Np + c] = t[n];
}

// Rows of a gradient, four columns a lane; with many parts (few rows) LANES lanes share
// out a column's, else a workgroup takes four rows.
template <int LANES>
__global__ __launch_bounds__(LANES > 1 ? 64 * LANES : 256) void sum_rows(VocabSum d) {
    constexpr int kRows = LANES > 1 ? 1 : 4;
    const int x = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = LANES > 1 ? x : 0;
    const int64_t i = (int64_t)blockIdx.x * kRows + (LANES > 1 ? 0 : x);
    const int col = 4 * (64 * (int)blockIdx.y + (threadIdx.x & 63));
    const bool mine = i < d.n && col < d.D;
    if (LANES == 1 && !mine) return;
    const int64_t c = !mine ? kRowOut : d.pos ? d.pos[i] : i;
    const float fill = c == kRowBad ? __builtin_nanf("") : 0.0f;
    float v[4] = {fill, fill, fill, fill};
    if (c >= 0) {
        const float* from = d.acc + (int64_t)c * d.Dp + col;
        int parts = d.parts;
        int64_t part = d.part;
        if (d.split.count) {
            const int rows = d.split.rows();
            parts = d.split.of(rows);
            part = (int64_t)rows * d.split.tile * d.Dp;
        }
        for (int s = lane; s < parts; s += 8 * LANES) {
            float4 a[8];
#pragma unroll
            for (int y = 0; y < 8; ++y)
                if (s + y * LANES < parts) a[y] = *reinterpret_cast<const float4*>(from + (s + y * LANES) * part);
#pragma unroll
            for (int y = 0; y < 8; ++y)
                if (s + y * LANES < parts) {
                    v[0] += a[y].x; v[1] += a[y].y; v[2] += a[y].z; v[3] += a[y].w;
                }
        }
    }
    if constexpr (LANES > 1) {
        __shared__ float4 sums[LANES][64];
        sums[lane][threadIdx.x & 63] = make_float4(v[0], v[1], v[2], v[3]);
        __syncthreads();
        if (lane > 0 || !mine) return;
#pragma unroll
        for (int y = 1; y < LANES; ++y) {
            const float4 a = sums[y][threadIdx.x];
            v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
        }
    }
    const int64_t at = i * d.ld + col;
    const int left = d.D - col;
    if (d.dtype == SSM_F32) store_dw(static_cast<float*>(d.out) + at, v, left, d.accumulate);
    else store_dw(static_cast<bf16_t*>(d.out) + at, v, left, d.accumulate);
}

unsigned blocks(int64_t n, int64_t per) { return (unsigned)((n + per - 1) / per); }
unsigned pack_blocks(const VocabPack& p) { return blocks((int64_t)p.n * ((p.width + 63) / 64 * 8), 256); }
int launched() { return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP; }

}  // namespace

int launch_vocab_rows(const VocabRows& r, uint32_t* err, hipStream_t stream) {
    if (r.K > 1 && r.N > 0) rows_state<<<blocks(r.N, 16), 256, 0, stream>>>(r, err);
    if (r.N <= 4096) rows_list<4><<<1, 1024, 0, stream>>>(r, err);
    else rows_list<16><<<1, 1024, 0, stream>>>(r, err);
    if (r.K > 1 && r.N > 0) rows_ids<<<blocks((int64_t)r.N * r.K, 256), 256, 0, stream>>>(r);
    return launched();
}

int launch_vocab_begin(const VocabBegin& v, int dtype, hipStream_t stream) {
    Begin b = {};
    auto turn_blocks = [](const VocabPack* p) { return p ? blocks(p->n, 64) * blocks(p->width, 64) : 0; };
    if (v.pack_h) b.pack_h = *v.pack_h;
    if (v.turn_h) b.turn_h = *v.turn_h;
    if (v.pack_w) b.pack_w = *v.pack_w;
    if (v.turn_w) b.turn_w = *v.turn_w;
    if (v.coef) b.coef = *v.coef;
    b.wide_h = is_wide(v.pack_h ? b.pack_h : b.turn_h);
    b.wide_w = is_wide(v.pack_w ? b.pack_w : b.turn_w);
    b.pack_h_end = v.pack_h ? pack_blocks(b.pack_h) : 0;
    b.pack_w_end = b.pack_h_end + (v.pack_w ? pack_blocks(b.pack_w) : 0);
    b.turn_h_end = b.pack_w_end + turn_blocks(v.turn_h);
    b.turn_w_end = b.turn_h_end + turn_blocks(v.turn_w);
    const unsigned grid = b.turn_w_end + (!v.coef ? 0 : blocks(b.coef.r.N, b.coef.r.logit ? 4 : 256));
    if (!grid) return SSM_OK;
    if (dtype == SSM_BF16) begin<1><<<grid, 256, 0, stream>>>(b);
    else begin<3><<<grid, 256, 0, stream>>>(b);
    return launched();
}

int launch_vocab_join(const VocabJoin& j, hipStream_t stream) {
    if (j.r.N <= 512) join_rows<256><<<j.r.N, 256, 0, stream>>>(j);
    else if (j.r.N <= 4096) join_rows<64><<<blocks(j.r.N, 4), 256, 0, stream>>>(j);
    else join_rows<8><<<blocks(j.r.N, 32), 256, 0, stream>>>(j);
    return launched();
}

int launch_vocab_few_begin(const VocabCoef& c, const VocabPack& turned, const VocabPack& packed, hipStream_t stream) {
    unsigned grid = kVocabFew / 4 + blocks(c.r.D, 64);
    if (c.r.terms == 1) {
        few_begin<1><<<grid, 256, 0, stream>>>(c, turned, packed, is_wide(turned));
    } else {
        grid += pack_blocks(packed);
        few_begin<3><<<grid, 256, 0, stream>>>(c, turned, packed, is_wide(turned));
    }
    return launched();
}

int launch_vocab_patch(const VocabPatch& p, hipStream_t stream) {
    const int groups = (int)blocks(p.r.N, 256);
    const unsigned grid = (unsigned)groups * p.r.K;
    if (p.terms == 1) patch_ids<1><<<grid, 256, 0, stream>>>(p, groups);
    else patch_ids<3><<<grid, 256, 0, stream>>>(p, groups);
    return launched();
}

int launch_vocab_sum(const VocabSum& d, hipStream_t stream) {
    if (d.parts > 16) sum_rows<16><<<dim3(d.n, blocks(d.D, 256)), 1024, 0, stream>>>(d);
    else sum_rows<1><<<dim3(blocks(d.n, 4), blocks(d.D, 256)), 256, 0, stream>>>(d);
    return launched();
}

}  // namespace ssm
