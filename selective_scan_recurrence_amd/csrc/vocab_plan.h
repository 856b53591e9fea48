// How the gradients of a loss over a vocabulary share out the card (host code, without
// HIP's headers).
#pragma once

#include <stdint.h>

#include <initializer_list>

namespace ssm {

constexpr int kVocabSplits = 64;  // parts of a gradient's sum, at most

inline int64_t vocab_tiles(int64_t m, int64_t n, int tile) { return (m + tile - 1) / tile * ((n + tile - 1) / tile); }

// Time until the last of nh workgroups of `a` us, and nw of `b` us after them in line,
// leave `places`.
inline double vocab_line_up(int64_t places, int64_t nh, double a, int64_t nw, double b) {
    const int64_t rounds = nh / places, late = nh % places, early = places - late;
    const double t0 = rounds * a, t1 = late ? t0 + a : t0;
    double t = t1;
    if (nw > 0) {
        // from the time that a perfect fit would take to the first with room for all
        const double least = (nw * b + early * t0 + late * t1) / places;
        int64_t j = (int64_t)((least - t0) / b);
        for (;; ++j) {
            const double e = t0 + j * b + 1e-6;
            const int64_t then = e > t1 ? (int64_t)((e - t1) / b) : 0;
            t = e;
            if (early * j + late * then >= nw) break;
            // the late places' next end, when it comes before the early ones'
            t = t1 + (then + 1) * b;
            if (t < e + b && early * j + late * (then + 1) >= nw) break;
        }
    }
    return t > t1 ? t : t1;
}

struct VocabParts {  // of the gradients' sums
    int d_h, d_w;
    int most;  // d_h: at most, with rows left out
    bool big;  // tiles of 256 x 256, else 128 x 128
};

// A launch of both sums, d_h [rows][width] over `vocab` and d_w [vocab][width] over the
// rows, or either alone: tiles, and parts of either sum, so that a long sum for few tiles
// (d_h of few rows, d_w of a small vocabulary) does not outlast all else, nor a last round
// of tiles leave most compute units idle.  f32, 1023 rows, width 771, vocabulary 10007: 204
// us, with a share of d_h for every compute unit 277.
inline VocabParts vocab_grads_parts(int64_t width, int64_t rows, int64_t vocab, bool d_h, bool d_w, int terms) {
    VocabParts best = {1, 1, 1, true};
    double least = 1e30;
    const int64_t n = d_h ? rows : 0, v = d_w ? vocab : 0;
    const int64_t steps_h = (vocab + 63) / 64, steps_w = (rows + 63) / 64, runs = terms == 3 ? 6 : 1;
    const int64_t most = steps_h / 4 < 1 ? 1 : steps_h / 4 < kVocabSplits ? steps_h / 4 : kVocabSplits;
    for (const bool big : {true, false}) {
        const int tile = big ? 256 : 128;
        const int64_t th = vocab_tiles(width, n, tile), tw = vocab_tiles(width, v, tile), places = big ? 256 : 512;
        // a workgroup's fair share of steps
        double share = (double)(th * steps_h + tw * steps_w) / places;
        if (share < 8) share = 8;
        const double even = th > 0 ? steps_h / share : 1;
        for (int x = 0; x < 8; ++x) {
            VocabParts p = {(int)(even * (0.5 + 0.25 * x) + 0.5), 1, (int)most, big};
            if (p.d_h < 1) p.d_h = 1;
            // the most parts are tried too, whatever share each then has (100 rows, width 64,
            // vocabulary 131072, bf16: 78 us a backward, in one part 2337)
            const bool last = p.d_h >= most;
            if (last) p.d_h = (int)most;
            for (int y = 0; y < 2; ++y) {
                if (y == 1) {
                    p.d_w = tw > 0 ? (int)(steps_w / share) : 1;
                    if (p.d_w <= 1) break;
                    if (p.d_w > kVocabSplits) p.d_w = kVocabSplits;
                }
                const int64_t nh = th * p.d_h, nw = tw * p.d_w;
                // alone on its compute unit a small tile's step takes 0.54 us
                const double step = big ? 1.48 : nh + nw <= 256 ? 0.54 : 0.88, rest = big ? 10.0 : 6.0;
                const double a = (step * runs * steps_h) / p.d_h + rest, b = (step * runs * steps_w) / p.d_w + rest;
                // parts of d_w take a kernel more; a part's read and write, at 4.5 TB/s
                const double kept = (p.d_h - 1) * (double)width * n + (p.d_w > 1 ? p.d_w * (double)width * v : 0.0);
                const double t = vocab_line_up(places, nh, a, nw, b) + (p.d_w > 1 ? 4 : 0) + 8e-6 / 4.5 * kept;
                if (t < least) {
                    least = t;
                    best = p;
                }
            }
            if (last) break;
        }
    }
    return best;
}

}  // namespace ssm
