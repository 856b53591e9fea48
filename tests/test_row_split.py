"""The weight gradient's split of its rows (csrc/row_split.h), compiled for the
host: the parts cover every row once for each size that the library takes, up
to the largest row count."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# first[i], last[i]: part i's rows, as the kernel forms them.  -fwrapv: what an
# overflow does there is what it does here.
SOURCE = """
#include "row_split.h"
extern "C" int split(int64_t M, int64_t W, int64_t O, int dtype, int* first, int* last) {
    const ssm::RowSplit s = ssm::split_rows(M, W, O, dtype);
    for (int i = 0; i < s.count; ++i) first[i] = i * s.rows, last[i] = ssm::part_end((int)M, s.rows, i);
    return s.count;
}
"""


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    d = tmp_path_factory.mktemp("split")
    (d / "split.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-O1", "-fwrapv", "-std=c++17", "-shared", "-fPIC",
                    "-I", os.path.join(ROOT, "selective_scan_recurrence_amd", "csrc"),
                    "-I", os.path.join(ROOT, "include"), str(d / "split.cpp"), "-o", str(d / "split.so")],
                   check=True)
    f = ctypes.CDLL(str(d / "split.so")).split
    f.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int] + [ctypes.c_void_p] * 2

    def parts(M, W, O, dtype):
        first, last = (ctypes.c_int * 512)(), (ctypes.c_int * 512)()
        n = f(M, W, O, dtype, first, last)
        assert 1 <= n <= 512
        return list(zip(first[:n], last[:n]))

    return parts


LARGEST = (1 << 31) - 1 - 1024


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("W,O", [(1, 1), (32, 16), (515, 130), (2560, 10576), (1 << 22, 3)])
def test_parts_cover_the_rows(split, dtype, W, O):
    for M in (0, 1, 63, 64, 65, 777, 8192, 100000, 2147450880, 2147450881, 2147467265, 2147482189, 2147482623,
              LARGEST - 64, LARGEST - 1, LARGEST):
        at = 0
        for first, last in split(M, W, O, dtype):
            assert first == at and (last > first or M == 0), (M, first, last)
            assert (last - first) % 64 == 0 or last == M
            at = last
        assert at == M
