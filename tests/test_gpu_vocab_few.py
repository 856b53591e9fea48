"""The losses over a vocabulary for up to 64 rows, whose kernels read W where it lies:
strides, d_W added to, and g's second term."""
import pytest
import torch

import vocab_ref as R
from test_gpu_vocab import compare, run
from vocab_few_ref import TwoTerms

pytestmark = pytest.mark.gpu

# one, two and four tiles of rows; widths of whole lines, of whole pieces and of neither
SIZES = [(1, 64, 300), (5, 130, 77), (16, 72, 1000), (31, 515, 640), (33, 128, 513), (64, 65, 300), (50, 2042, 129)]


@pytest.mark.parametrize("pad_h,pad_w", [(0, 1), (1, 0), (8, 64), (3, 8)])
@pytest.mark.parametrize("io,dw", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("n,d,v", SIZES)
def test_strides(n, d, v, io, dw, pad_h, pad_w):
    """Slices of wider tensors; what lies behind their rows stays as it was."""
    t = R.problem(n + d, n, d, v, io, out=0.2 if n > 4 else 0.0)
    compare(t, io, run(t, io, dw=dw, pad_h=pad_h, pad_w=pad_w), dw=dw)


@pytest.mark.parametrize("pad_w", [0, 3])
@pytest.mark.parametrize("top", [0, 4])
@pytest.mark.parametrize("io,dw", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("n,d,v", SIZES)
def test_accumulates(n, d, v, io, dw, top, pad_w):
    t = R.problem(n + d + top, n, d, v, io, top=top, out=0.2 if n > 4 else 0.0)
    d_w0 = (0.1 * torch.randn(v, d, generator=torch.Generator().manual_seed(n))).to(R.DTYPES[dw])
    compare(t, io, run(t, io, dw=dw, pad_w=pad_w, d_w0=d_w0), dw=dw, d_w0=d_w0)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_no_rows_add_nothing(io):
    """What the weight gradient held stays, also behind its rows."""
    d_w0 = torch.randn(300, 65, generator=torch.Generator().manual_seed(1))
    t = {"h": torch.zeros(0, 65), "w": torch.zeros(300, 65), "target": torch.zeros(0, dtype=torch.int32),
         "d_loss": torch.zeros(0)}
    assert torch.equal(run(t, io, d_w0=d_w0, pad_w=5)["d_w"].cpu(), d_w0)


@pytest.mark.parametrize("n", [1, 7, 33, 64])
@pytest.mark.parametrize("d", [8, 64, 130])
def test_g_has_two_terms(n, d):
    t = R.problem(n + d, n, d, 300, "bf16")
    R.check("d_w", run(t, "bf16", dw="f32")["d_w"],
            *TwoTerms(t["h"], t["w"], "bf16", target=t["target"]).d_w(t["d_loss"]))
