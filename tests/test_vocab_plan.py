"""How the gradients of the losses over a vocabulary are shared out
(csrc/vocab_plan.h), compiled for the host: no workgroup's sum is much longer than
a fair share, or than the most parts leave it."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = """
#include "vocab_plan.h"
extern "C" void plan(int64_t width, int64_t rows, int64_t vocab, int d_h, int d_w, int terms, int* out) {
    const ssm::VocabParts p = ssm::vocab_grads_parts(width, rows, vocab, d_h, d_w, terms);
    out[0] = p.d_h, out[1] = p.d_w, out[2] = p.most, out[3] = p.big;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC",
                    "-I", os.path.join(ROOT, "selective_scan_recurrence_amd", "csrc"), str(d / "plan.cpp"),
                    "-o", str(d / "plan.so")], check=True)
    f = ctypes.CDLL(str(d / "plan.so")).plan
    f.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int] * 3 + [ctypes.c_void_p]

    def parts(*args):
        out = (ctypes.c_int * 4)()
        f(*args, out)
        return tuple(out)

    return parts


def _ceil(a, b):
    return -(-a // b)


def _check(plan, width, rows, vocab, d_h, d_w, terms):
    n_h, n_w, most, big = plan(width, rows, vocab, d_h, d_w, terms)
    case = (width, rows, vocab, d_h, d_w, terms, n_h, n_w, most, big)
    steps_h, steps_w = _ceil(vocab, 64), _ceil(rows, 64)
    assert most == max(1, min(64, steps_h // 4)) and 1 <= n_h <= most and 1 <= n_w <= max(1, min(64, steps_w)), case
    tile = 256 if big else 128
    tiles_h = _ceil(width, tile) * _ceil(rows, tile) if d_h else 0
    tiles_w = _ceil(width, tile) * _ceil(vocab, tile) if d_w else 0
    share = max(8, (tiles_h * steps_h + tiles_w * steps_w) / (256 if big else 512))
    # the fewest parts that are tried are half of what a share for each takes, rounded
    if d_h:
        assert steps_h / n_h <= max(3 * share, steps_h / most), case


@pytest.mark.parametrize("width,rows,vocab,d_w", [
    (64, 100, 65536, 1), (64, 100, 66000, 1), (64, 100, 131072, 1), (64, 65, 1 << 20, 1), (128, 128, 131072, 1),
    (256, 100, 262144, 0), (200, 256, 262144, 0), (1, 65, 1 << 24, 0), (2560, 16384, 32768, 1), (65536, 65, 300, 1),
])
@pytest.mark.parametrize("terms", [1, 3])
def test_a_long_vocabulary_is_shared_out(plan, width, rows, vocab, d_w, terms):
    _check(plan, width, rows, vocab, 1, d_w, terms)


def test_drawn_sizes(plan):
    rng = random.Random(3)

    def spread(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    for _ in range(3000):
        d_h, d_w = rng.choice([(1, 1), (1, 0), (0, 1)])
        _check(plan, spread(1, 65536), spread(65, 1 << 20), spread(1, 1 << 24), d_h, d_w, rng.choice([1, 3]))
