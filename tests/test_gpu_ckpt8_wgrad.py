"""ssm_ckpt8_wgrad on the GPU against the float64 product of dy with the
values the checkpoint holds: tile ends in every direction, few and many rows,
split sums, strides, accumulation."""
import pytest
import torch

import block_ref as R
from selective_scan_recurrence_amd import ops

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1, 1), (1, 32, 16), (2, 33, 17), (31, 64, 64), (32, 100, 130), (33, 128, 256), (64, 256, 128),
          (65, 515, 70), (100, 31, 300), (257, 260, 257), (777, 515, 130), (1000, 48, 48), (4100, 64, 80),
          (2048, 256, 512), (300, 1024, 776)]


def _case(rows, width, n_out, io, pad=0, seed=0):
    x = R.draw(seed + 1, rows, width)
    dy = R.draw(seed + 2, rows, n_out).to(R.DTYPES[io])
    ck = ops.ckpt8_pack(x.cuda())
    back = ops.ckpt8_unpack(ck, rows, width, io="f32").double().cpu()
    return dy, R.strided(dy.float(), pad, R.DTYPES[io]), ck, dy.double().t() @ back, \
        dy.double().abs().t() @ back.abs()


def _bound(rows):
    # exact products; at most one rounding a row added in sequence, and some
    # for joining partial sums
    return rows + 40


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,width,n_out", SHAPES)
def test_product(rows, width, n_out, io):
    pad = (rows + width) % 3 * 4
    _, dyd, ck, want, mag = _case(rows, width, n_out, io, pad, seed=rows)
    out = torch.full((n_out * width + 64,), float("nan"), device="cuda")
    got = ops.ckpt8_wgrad(dyd, ck, width, dw=out[:n_out * width].view(n_out, width))
    R.check("dw", got, want, mag, "f32", _bound(rows))
    assert torch.isnan(out[n_out * width:]).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,width,n_out", [(40, 70, 33), (3000, 96, 64), (300, 520, 260)])
def test_accumulate(rows, width, n_out, io):
    _, dyd, ck, want, mag = _case(rows, width, n_out, io)
    first = R.draw(9, n_out, width)
    dw = first.cuda()
    ops.ckpt8_wgrad(dyd, ck, width, dw=dw, accumulate=True)
    R.check("dw", dw, want + first.double(), mag + first.double().abs(), "f32", _bound(rows))


def test_odd_row_stride():
    """dy rows at odd element offsets of a wider matrix."""
    rows, width, n_out = 200, 128, 192
    dy = R.draw(2, rows, n_out).bfloat16()
    wide = torch.zeros(rows, n_out + 77, dtype=torch.bfloat16, device="cuda")
    wide[:, 33:33 + n_out] = dy.cuda()
    ck = ops.ckpt8_pack(R.draw(1, rows, width).cuda())
    back = ops.ckpt8_unpack(ck, rows, width, io="f32").double().cpu()
    got = ops.ckpt8_wgrad(wide[:, 33:33 + n_out], ck, width)
    R.check("dw", got, dy.double().t() @ back, dy.double().abs().t() @ back.abs(), "f32", _bound(rows))


def test_no_rows():
    dy = torch.zeros(0, 40, dtype=torch.bfloat16, device="cuda")
    ck = torch.empty(0, dtype=torch.uint8, device="cuda")
    nan = torch.full((40, 64), float("nan"), device="cuda")
    assert not ops.ckpt8_wgrad(dy, ck, 64, dw=nan).any()
    ones = torch.ones(40, 64, device="cuda")
    assert bool((ops.ckpt8_wgrad(dy, ck, 64, dw=ones, accumulate=True) == 1).all())


def test_wide_scales():
    """Blocks of very different scales, and f32 gradients that need all 24 bits."""
    rows, width, n_out = 96, 96, 64
    x = R.draw(1, rows, width) * torch.logspace(-12, 6, rows).unsqueeze(1)
    dy = R.draw(2, rows, n_out) * (1 + 2.0 ** -20)
    ck = ops.ckpt8_pack(x.cuda())
    back = ops.ckpt8_unpack(ck, rows, width, io="f32").double().cpu()
    got = ops.ckpt8_wgrad(dy.cuda(), ck, width)
    R.check("dw", got, dy.double().t() @ back, dy.double().abs().t() @ back.abs(), "f32", _bound(rows))


def test_largest_gradients():
    """f32 gradients up to the largest value, which no part of their split may
    pass, and ones whose low parts are subnormal."""
    top = torch.finfo(torch.float32).max
    dy = torch.tensor([[top, -top, 1.0, 2.0 ** -100 * (1 + 2.0 ** -23)]] * 3)
    x = torch.zeros(3, 32)
    x[0] = 0.5
    got = ops.ckpt8_wgrad(dy.cuda(), ops.ckpt8_pack(x.cuda()), 32).double().cpu()
    want = (dy[0].double() * 0.5).unsqueeze(1).expand(4, 32)
    assert torch.equal(got[:3], want[:3])
    assert ((got[3] - want[3]).abs() <= want[3] * 2.0 ** -23).all()


def test_nan_stays_in_its_column():
    x, dy = R.draw(1, 50, 96), R.draw(2, 50, 40)
    x[7, 5] = float("nan")
    dy[9, 3] = float("inf")
    got = ops.ckpt8_wgrad(dy.cuda(), ops.ckpt8_pack(x.cuda()), 96).cpu()
    bad = ~torch.isfinite(got)
    assert bad[:, 5].all() and bad[3].all()
    bad[:, 5] = bad[3] = False
    assert not bad.any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_repeats_bitwise(io):
    _, dyd, ck, _, _ = _case(5000, 160, 96, io)
    first = ops.ckpt8_wgrad(dyd, ck, 160)
    for _ in range(3):
        assert torch.equal(ops.ckpt8_wgrad(dyd, ck, 160), first)
