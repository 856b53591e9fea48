// The C ABI of the losses over a vocabulary (declared in include/ssm.h): argument
// checks on the host, the workspace's layout, and the launches of a call.
// Nothing here reads device memory or allocates.
#include <math.h>

#include <initializer_list>

#include "vocab.h"

namespace ssm {
namespace {

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }  // NULL passes
bool known(int32_t dtype) { return dtype == SSM_F32 || dtype == SSM_BF16; }
size_t size_of(int32_t dtype) { return dtype == SSM_BF16 ? 2 : 4; }
int64_t round_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// A row of bf16 values whose length is a multiple of 4 KB gets 512 bytes more: such
// rows start in the same channels of the caches (a gradient's products of 16384 x 16384
// rows, width 2560: 2070 us, without 2140).
int64_t off_channels(int64_t v) { return v % 2048 ? v : v + 256; }

constexpr int kMostVocab = 1 << 24;

struct VocabShape {
    int N, D, V, K, top;
    // Bf16 terms of g.  One with bf16 tensors, as their results are rounded: a second would
    // double the 4.2 ms that both products take in a step's 8.9 (16384 rows, width 2560,
    // vocabulary 32768).  Up to 64 rows, where W's bytes bound the products, two.
    int g_terms;
    int64_t ld_h, ld_w;
    int io, dw, terms;
    float scale, top_scale;
    bool accumulate;
};

int check(const ssm_vocab_desc* d, VocabShape* out) {
    if (!d) return SSM_ERR_NULL;
    if (!known(d->io_dtype) || !known(d->dw_dtype)) return SSM_ERR_DTYPE;
    if (d->reserved != 0 || (d->flags & ~(uint32_t)SSM_VOCAB_ACCUMULATE)) return SSM_ERR_SHAPE;
    if (d->n_rows < 0 || d->n_rows > 1 << 21 || d->width < 1 || d->width > 1 << 16 || d->n_vocab < 1 ||
        d->n_vocab > kMostVocab || d->n_top < 0 || d->n_top > 1024)
        return SSM_ERR_SHAPE;
    // a launch has under 2^32 lanes, and h is packed 8 values a lane
    if (d->n_rows * d->width > (int64_t)1 << 34) return SSM_ERR_SHAPE;
    VocabShape s;
    s.N = (int)d->n_rows; s.D = (int)d->width; s.V = (int)d->n_vocab;
    s.top = (int)d->n_top; s.K = s.top ? s.top : 1;
    s.ld_h = d->ld_h ? d->ld_h : s.D;
    s.ld_w = d->ld_w ? d->ld_w : s.D;
    if (s.ld_h < s.D || s.ld_w < s.D || s.ld_h > 1 << 22 || s.ld_w > 1 << 22) return SSM_ERR_SHAPE;
    // the logits carry scale log2 e
    if (!isfinite(d->scale * kLog2e) || !isfinite(d->top_scale)) return SSM_ERR_SHAPE;
    s.io = d->io_dtype; s.dw = d->dw_dtype; s.terms = s.io == SSM_BF16 ? 1 : 3;
    s.g_terms = s.terms == 3 ? 3 : s.N <= kVocabFew ? 2 : 1;
    if (s.io == SSM_F32 && s.dw == SSM_BF16) return SSM_ERR_UNSUPPORTED;
    s.scale = d->scale; s.top_scale = d->top_scale;
    s.accumulate = d->flags & SSM_VOCAB_ACCUMULATE;
    *out = s;
    return SSM_OK;
}

// Where a call keeps what in its workspace, and the vocabulary's pieces.  A
// piece's tensors take up to 1.25 GiB: with 16384 rows in bf16 that is 16384
// of the vocabulary, long enough a sum that adding to d_h once a piece costs
// little (a piece's two gradients take 2 ms, the addition 0.07).
struct Plan {
    int64_t Np, Kd, piece, ld;  // ld: row stride of what has the piece as columns
    int pieces;
    VocabParts parts;  // backward: set by the call
    bool few, packed;  // W goes through the workspace
    size_t count, rows, pos, kid, h, part, state, slog, w, ht, wt, g, gt, lse2, coef, at, acc, acc_w, bytes;
};

constexpr int64_t kPieceBytes = (int64_t)5 << 28;

VocabParts parts_of(const VocabShape& s, const Plan& p, bool d_h, bool d_w) {
    if (p.few) return {vocab_few_splits(p.piece, s.D), 1, 1, false};
    return vocab_grads_parts(s.D, s.N, p.piece, d_h, d_w, s.terms);
}

Plan plan_of(const VocabShape& s, bool backward, bool packed) {
    Plan p;
    p.few = s.N <= kVocabFew;
    p.Np = p.few ? kVocabFew : off_channels(round_up(s.N, kVocabTile));
    p.Kd = round_up(s.D, kVocabStep);
    p.packed = packed && !p.few;
    packed = p.packed;
    const int64_t T = s.terms, V = round_up(s.V, kVocabTile);
    // bytes a vocabulary entry of a piece
    int64_t each = packed ? T * p.Kd * 2 : 0;
    each += backward ? 4 * s.g_terms * p.Np + (p.few ? 0 : 2 * T * p.Kd) : p.Np / (p.few ? 4 : 8);
    int64_t most = kPieceBytes / each / kVocabTile * kVocabTile;
    if (most < kVocabTile) most = kVocabTile;
    p.pieces = (int)((V + most - 1) / most);
    p.piece = round_up((V + p.pieces - 1) / p.pieces, kVocabTile);
    p.pieces = (int)((V + p.piece - 1) / p.piece);
    p.ld = p.few ? p.piece : off_channels(p.piece);

    size_t at = 0;
    auto take = [&](int64_t n) {
        const size_t here = at;
        at += (size_t)round_up(n, 256);
        return here;
    };
    p.count = take(4);
    p.rows = take(p.Np * 4);
    p.pos = take(p.Np * 4);
    p.kid = take(p.Np * s.K * 4);
    p.h = p.few && T == 1 ? 0 : take(T * p.Np * p.Kd * 2);
    p.w = packed ? take(T * p.piece * p.Kd * 2) : 0;
    if (backward) {
        p.ht = take(T * s.D * p.Np * 2);
        p.wt = p.few ? 0 : take(T * s.D * p.ld * 2);
        p.g = take(s.g_terms * p.Np * p.ld * 2);
        p.gt = take(s.g_terms * p.Np * p.ld * 2);
        p.lse2 = take(p.Np * 4);
        p.coef = take(p.Np * 4);
        p.at = take(p.Np * s.K * 4);
        // of the three calls (both gradients, either alone) the one that takes the most
        int64_t acc = 0, acc_w = 0;
        for (int x = 1; x < 4; ++x) {
            const VocabParts n = parts_of(s, p, x & 1, x & 2);
            if (n.d_h > acc) acc = n.d_h;
            if (n.d_w > acc_w) acc_w = n.d_w;
        }
        p.acc = take(acc * p.Np * p.Kd * 4);
        p.acc_w = acc_w > 1 ? take(acc_w * p.piece * p.Kd * 4) : 0;
    } else {
        p.part = take(p.piece / (p.few ? 32 : 64) * p.Np * 8);
        p.state = take(p.Np * 8);
        p.slog = take(p.Np * s.K * 4);
    }
    p.bytes = at;
    return p;
}

// W's rows are read where they are when they are whole pieces of 128 bytes
bool reads_w(const VocabShape& s, const void* w) {
    return s.io == SSM_BF16 && s.D % kVocabStep == 0 && s.ld_w % 8 == 0 && aligned(w, 16);
}

size_t workspace_bytes(const VocabShape& s, bool backward) {
    // w's address is not known here: it may need the packed form
    const size_t packed = plan_of(s, backward, true).bytes, direct = plan_of(s, backward, false).bytes;
    size_t n = packed > direct ? packed : direct;
    if (backward) {
        const size_t f = workspace_bytes(s, false);
        n = n > f ? n : f;
    }
    return n;
}

struct Call {
    VocabShape s;
    Plan p;
    VocabRows r;
    const void *h, *w;
    char* ws;
    hipStream_t stream;
    template <typename T>
    T* at(size_t off) const { return reinterpret_cast<T*>(ws + off); }
};

Call make_call(const VocabShape& s, bool backward, const void* h, const void* w, const int32_t* id,
               const float* logit, const float* top_lse, void* ws, hipStream_t stream) {
    Call c = {s, plan_of(s, backward, !reads_w(s, w)), {}, h, w, static_cast<char*>(ws), stream};
    c.r = {s.N, s.D, s.V, s.K, (int)c.p.Np, s.terms, id, logit, top_lse, s.top_scale,
           c.at<int32_t>(c.p.count), c.at<int32_t>(c.p.rows), c.at<int32_t>(c.p.pos), c.at<int32_t>(c.p.kid)};
    return c;
}

#define RUN(x)                  \
    do {                        \
        const int rc_ = (x);    \
        if (rc_) return rc_;    \
    } while (0)

VocabPack pack_h(const Call& c, size_t to, int64_t plane) {
    return {c.h, c.s.ld_h, c.s.io, c.s.D, c.s.N, 0, c.r.rows, c.r.count, c.at<uint16_t>(to), c.p.Np, plane};
}

VocabPack pack_w(const Call& c, int64_t v0, int n, size_t to, int64_t plane) {
    return {c.w, c.s.ld_w, c.s.io, c.s.D, n, v0, nullptr, nullptr, c.at<uint16_t>(to), c.p.ld, plane};
}

// What comes before a piece's logits: W's rows packed unless they are read where they
// are, and turned for d_h; before the first piece also `first`.
int begin_piece(const Call& c, int x, int64_t v0, int n, bool turn, const VocabBegin& first) {
    VocabBegin b = x == 0 ? first : VocabBegin();
    const VocabPack packed = pack_w(c, v0, n, c.p.w, c.p.piece * c.p.Kd);
    const VocabPack turned = pack_w(c, v0, n, c.p.wt, c.s.D * c.p.ld);
    if (c.p.packed) b.pack_w = &packed;
    if (turn) b.turn_w = &turned;
    return launch_vocab_begin(b, c.s.io, c.stream);
}

// the operands of a piece's logits
VocabGemm logits(const Call& c, int64_t v0, int n) {
    VocabGemm g = {};
    if (c.p.packed) {
        g.a = c.at<uint16_t>(c.p.w);
        g.a_plane = c.p.piece * c.p.Kd;
        g.lda = c.p.Kd;
    } else {
        g.a = static_cast<const uint16_t*>(c.w) + v0 * c.s.ld_w;
        g.lda = c.s.ld_w;
    }
    g.b = c.at<uint16_t>(c.p.h);
    g.b_plane = c.p.Np * c.p.Kd;
    g.ldb = c.p.Kd;
    g.m = n; g.n = c.s.N; g.k = (int)c.p.Kd;
    g.count = c.r.count;
    g.Np = c.p.Np;
    g.scale2 = c.s.scale * kLog2e;
    g.v0 = (int)v0; g.K = c.s.K; g.ld_g = c.p.ld;
    g.kid = c.r.kid;
    return g;
}

int forward_few(const Call& c, float* loss, float* lse, float* logq, uint32_t* err);

int forward(const Call& c, float* loss, float* lse, float* logq, uint32_t* err) {
    const Plan& p = c.p;
    if (p.few) return forward_few(c, loss, lse, logq, err);
    RUN(launch_vocab_rows(c.r, err, c.stream));
    const VocabPack packed = pack_h(c, p.h, p.Np * p.Kd);
    VocabBegin first;
    first.pack_h = &packed;
    for (int x = 0; x < p.pieces; ++x) {
        const int64_t v0 = x * p.piece;
        const int n = (int)(c.s.V - v0 < p.piece ? c.s.V - v0 : p.piece);
        RUN(begin_piece(c, x, v0, n, false, first));
        VocabGemm g = logits(c, v0, n);
        g.part = c.at<float2>(p.part);
        g.slog = c.at<float>(p.slog);
        RUN(launch_vocab_logits_fwd(g, c.s.terms, c.stream));
        RUN(launch_vocab_join({c.r, g.part, vocab_parts(g, c.s.terms), c.at<float2>(p.state), x == 0,
                               x == p.pieces - 1, g.slog, loss, lse, logq, nullptr}, c.stream));
    }
    return SSM_OK;
}

VocabFew few_of(const Call& c) {
    VocabFew f = {};
    f.r = c.r;
    f.h = c.h; f.w = c.w;
    f.ld_h = c.s.ld_h; f.ld_w = c.s.ld_w;
    f.scale2 = c.s.scale * kLog2e;
    f.P = (int)c.p.piece;
    if (c.s.terms == 3) f.hp = c.at<uint16_t>(c.p.h);
    return f;
}

// h where rows keep their places
VocabPack placed_h(const Call& c, size_t to, int64_t plane) {
    VocabPack p = pack_h(c, to, plane);
    p.rows = p.count = nullptr;
    return p;
}

// a piece takes the whole vocabulary
static_assert(((int64_t)kMostVocab * kVocabFew / 4) <= kPieceBytes, "");
int forward_few(const Call& c, float* loss, float* lse, float* logq, uint32_t* err) {
    const Plan& p = c.p;
    VocabFew f = few_of(c);
    f.r.pos = nullptr;
    f.part = c.at<float2>(p.part);
    f.slog = c.at<float>(p.slog);
    const int tile = vocab_few_part(c.r);
    if (c.s.terms == 3) {
        const VocabPack packed = placed_h(c, p.h, p.Np * p.Kd);
        VocabBegin b;
        b.pack_h = &packed;
        RUN(launch_vocab_begin(b, c.s.io, c.stream));
    }
    RUN(launch_vocab_few_logits(f, false, c.stream));
    return launch_vocab_join({f.r, f.part, (c.s.V + tile - 1) / tile, nullptr, true, true, f.slog, loss, lse, logq, err},
                             c.stream);
}

// the product for d_w of a piece [v0, v0 + n), or of its sum's parts
VocabGemm product_w(const Call& c, int64_t v0, int n, void* d_w) {
    const Plan& p = c.p;
    VocabGemm g = {};
    g.a = c.at<uint16_t>(p.ht); g.a_plane = c.s.D * p.Np; g.lda = p.Np;
    g.b = c.at<uint16_t>(p.gt); g.b_plane = p.Np * p.ld; g.ldb = p.Np;
    g.m = c.s.D; g.n = d_w ? n : 0;
    g.splits = p.parts.d_w;
    if (p.parts.d_w > 1) {
        g.out = c.at<float>(p.acc_w); g.ld_out = p.Kd; g.out_part = p.piece * p.Kd;
        g.out_dtype = SSM_F32;
    } else {
        g.out = static_cast<char*>(d_w) + v0 * c.s.ld_w * (int64_t)size_of(c.s.dw); g.ld_out = c.s.ld_w;
        g.out_dtype = c.s.dw; g.accumulate = c.s.accumulate;
    }
    return g;
}

int join_d_w(const Call& c, int64_t v0, int n, void* d_w) {
    const Plan& p = c.p;
    return launch_vocab_sum({c.at<float>(p.acc_w), p.piece * p.Kd, p.parts.d_w, (int)p.Kd, {}, nullptr, n, c.s.D,
                             c.s.dw, static_cast<char*>(d_w) + v0 * c.s.ld_w * (int64_t)size_of(c.s.dw), c.s.ld_w,
                             c.s.accumulate}, c.stream);
}

VocabSplit split_of(const Call& c) {
    return {c.r.count, c.s.N, c.p.parts.big ? 256 : 128, c.p.parts.d_h, c.p.parts.most};
}

int join_d_h(const Call& c, void* d_h) {
    const Plan& p = c.p;
    VocabSum d = {c.at<float>(p.acc), p.Np * p.Kd, p.parts.d_h, (int)p.Kd, {}, c.r.pos, c.s.N, c.s.D, c.s.io,
                  d_h, c.s.ld_h, false};
    if (!p.few) d.split = split_of(c);
    return launch_vocab_sum(d, c.stream);
}

VocabCoef factors(const Call& c, const float* logq, const float* loss, const float* lse, const float* d_loss,
                  const float* d_lse) {
    return {c.r, logq, loss, lse, d_loss, d_lse, c.s.scale, c.at<float>(c.p.lse2), c.at<float>(c.p.coef),
            c.at<float>(c.p.at)};
}

int backward_few(const Call& c, const VocabCoef& f, void* d_h, void* d_w) {
    const Plan& p = c.p;
    const VocabShape& s = c.s;
    RUN(launch_vocab_few_begin(f, placed_h(c, p.ht, s.D * p.Np), placed_h(c, p.h, p.Np * p.Kd), c.stream));
    VocabFew few = few_of(c);
    few.lse2 = f.lse2; few.coef = f.coef; few.at = f.at;
    few.g = c.at<uint16_t>(p.g); few.gt = c.at<uint16_t>(p.gt);
    few.ht = c.at<uint16_t>(p.ht);
    few.dw_dtype = s.dw; few.accumulate = s.accumulate;
    few.acc = c.at<float>(p.acc); few.splits = p.parts.d_h;
    for (int x = 0; x < p.pieces; ++x) {
        few.v0 = (int)(x * p.piece);
        few.first = x == 0;
        if (s.N > 0) RUN(launch_vocab_few_logits(few, true, c.stream));
        if (d_h && s.N > 0) RUN(launch_vocab_few_d_h(few, c.stream));
        if (d_w) {
            few.d_w = static_cast<char*>(d_w) + few.v0 * s.ld_w * (int64_t)size_of(s.dw);
            RUN(launch_vocab_few_d_w(few, c.stream));
        }
    }
    return d_h && s.N > 0 ? join_d_h(c, d_h) : SSM_OK;
}

int backward(const Call& c, const float* logq, const float* loss, const float* lse, const float* d_loss,
             const float* d_lse, void* d_h, void* d_w) {
    const Plan& p = c.p;
    const VocabShape& s = c.s;
    if (!d_h && !d_w) return SSM_OK;
    const VocabCoef f = factors(c, logq, loss, lse, d_loss, d_lse);
    if (p.few) return backward_few(c, f, d_h, d_w);
    RUN(launch_vocab_rows(c.r, nullptr, c.stream));
    const VocabPack packed = pack_h(c, p.h, p.Np * p.Kd), turned = pack_h(c, p.ht, s.D * p.Np);
    VocabBegin first;
    first.pack_h = &packed;
    if (d_w) first.turn_h = &turned;
    first.coef = &f;
    uint16_t *g = c.at<uint16_t>(p.g), *gt = c.at<uint16_t>(p.gt);
    for (int x = 0; x < p.pieces; ++x) {
        const int64_t v0 = x * p.piece;
        const int n = (int)(s.V - v0 < p.piece ? s.V - v0 : p.piece);
        RUN(begin_piece(c, x, v0, n, d_h != nullptr, first));
        VocabGemm l = logits(c, v0, n);
        l.lse2 = f.lse2;
        l.coef = f.coef;
        l.g = g;
        l.gt = gt;
        RUN(launch_vocab_logits_bwd(l, s.terms, c.stream));
        RUN(launch_vocab_patch({c.r, f.at, (int)v0, n, s.g_terms, p.ld, p.Np * p.ld, g, gt}, c.stream));
        VocabGemm gh = {};
        gh.a = c.at<uint16_t>(p.wt); gh.a_plane = s.D * p.ld; gh.lda = p.ld;
        gh.b = g; gh.b_plane = p.Np * p.ld; gh.ldb = p.ld;
        gh.m = s.D; gh.n = d_h ? s.N : 0; gh.k = (int)round_up(n, kVocabStep);
        gh.count = c.r.count; gh.Np = p.Np;
        gh.out = c.at<float>(p.acc); gh.ld_out = p.Kd; gh.split = split_of(c);
        gh.accumulate = x > 0;
        RUN(launch_vocab_grads(gh, product_w(c, v0, n, d_w), s.terms, p.parts.big, c.stream));
        if (d_w && p.parts.d_w > 1) RUN(join_d_w(c, v0, n, d_w));
    }
    return d_h ? join_d_h(c, d_h) : SSM_OK;
}

// what every call checks of its tensors
int check_call(const VocabShape& s, bool backward, const void* h, const void* w, const int32_t* id,
               const void* ws, size_t bytes) {
    if (!w || !ws || (s.N > 0 && (!h || !id))) return SSM_ERR_NULL;
    if (bytes < workspace_bytes(s, backward)) return SSM_ERR_WORKSPACE;
    const size_t es = size_of(s.io);
    return aligned(h, es) && aligned(w, es) && aligned(id, 4) && aligned(ws, 256) ? SSM_OK : SSM_ERR_ALIGN;
}

bool all_aligned(size_t a, std::initializer_list<const void*> list) {
    for (const void* p : list)
        if (!aligned(p, a)) return false;
    return true;
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" {

size_t ssm_vocab_workspace_bytes(const ssm_vocab_desc* desc, int backward) {
    VocabShape s;
    return check(desc, &s) == SSM_OK ? workspace_bytes(s, backward != 0) : 0;
}

int ssm_vocab_ce_fwd(const ssm_vocab_desc* desc, const void* h, const void* w, const int32_t* target,
                     float* loss, float* lse, uint32_t* err, void* workspace, size_t workspace_bytes,
                     ssm_stream_t stream) {
    VocabShape s;
    RUN(check(desc, &s));
    if (s.top) return SSM_ERR_SHAPE;
    RUN(check_call(s, false, h, w, target, workspace, workspace_bytes));
    if (!all_aligned(4, {loss, lse, err})) return SSM_ERR_ALIGN;
    if (s.N == 0) return SSM_OK;
    const Call c = make_call(s, false, h, w, target, nullptr, nullptr, workspace, static_cast<hipStream_t>(stream));
    return forward(c, loss, lse, nullptr, err);
}

int ssm_vocab_ce_bwd(const ssm_vocab_desc* desc, const void* h, const void* w, const int32_t* target,
                     const float* loss, const float* lse, const float* d_loss, const float* d_lse,
                     void* d_h, void* d_w, void* workspace, size_t workspace_bytes, ssm_stream_t stream) {
    VocabShape s;
    RUN(check(desc, &s));
    if (s.top) return SSM_ERR_SHAPE;
    RUN(check_call(s, true, h, w, target, workspace, workspace_bytes));
    if (s.N > 0 && (!loss || !lse || !d_loss)) return SSM_ERR_NULL;
    if (!all_aligned(4, {loss, lse, d_loss, d_lse}) || !aligned(d_h, size_of(s.io)) || !aligned(d_w, size_of(s.dw)))
        return SSM_ERR_ALIGN;
    Call c = make_call(s, true, h, w, target, nullptr, nullptr, workspace, static_cast<hipStream_t>(stream));
    c.p.parts = parts_of(s, c.p, d_h, d_w);
    return backward(c, nullptr, loss, lse, d_loss, d_lse, d_h, d_w);
}

int ssm_vocab_kd_fwd(const ssm_vocab_desc* desc, const void* h, const void* w, const int32_t* top_id,
                     const float* top_logit, const float* top_lse, float* loss, float* lse, float* logq,
                     uint32_t* err, void* workspace, size_t workspace_bytes, ssm_stream_t stream) {
    VocabShape s;
    RUN(check(desc, &s));
    if (!s.top) return SSM_ERR_SHAPE;
    RUN(check_call(s, false, h, w, top_id, workspace, workspace_bytes));
    if (s.N > 0 && !top_logit) return SSM_ERR_NULL;
    if (!all_aligned(4, {top_logit, top_lse, loss, lse, logq, err})) return SSM_ERR_ALIGN;
    if (s.N == 0) return SSM_OK;
    const Call c = make_call(s, false, h, w, top_id, top_logit, top_lse, workspace, static_cast<hipStream_t>(stream));
    return forward(c, loss, lse, logq, err);
}

int ssm_vocab_kd_bwd(const ssm_vocab_desc* desc, const void* h, const void* w, const int32_t* top_id,
                     const float* top_logit, const float* top_lse, const float* logq, const float* lse,
                     const float* d_loss, const float* d_lse, void* d_h, void* d_w, void* workspace,
                     size_t workspace_bytes, ssm_stream_t stream) {
    VocabShape s;
    RUN(check(desc, &s));
    if (!s.top) return SSM_ERR_SHAPE;
    RUN(check_call(s, true, h, w, top_id, workspace, workspace_bytes));
    if (s.N > 0 && (!top_logit || !logq || !lse || !d_loss)) return SSM_ERR_NULL;
    if (!all_aligned(4, {top_logit, top_lse, logq, lse, d_loss, d_lse}) || !aligned(d_h, size_of(s.io)) ||
        !aligned(d_w, size_of(s.dw)))
        return SSM_ERR_ALIGN;
    Call c = make_call(s, true, h, w, top_id, top_logit, top_lse, workspace, static_cast<hipStream_t>(stream));
    c.p.parts = parts_of(s, c.p, d_h, d_w);
    return backward(c, logq, nullptr, lse, d_loss, d_lse, d_h, d_w);
}

}  // extern "C"
