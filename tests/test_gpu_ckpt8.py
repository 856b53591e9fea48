"""ssm_ckpt8_pack and ssm_ckpt8_unpack on the GPU: codes and scale bytes equal
the search of tests/block_ref.py bit for bit, and reading back is exact."""
import pytest
import torch

import block_ref as R
from selective_scan_recurrence_amd import ops

pytestmark = pytest.mark.gpu


def _split(ck, rows, width):
    w32 = -(-width // 32) * 32
    ck = ck.cpu()
    return ck[:rows * w32].view(rows, w32), ck[rows * w32:].view(rows, w32 // 32)


def _check(x, t):
    """x: CPU values of t, the device tensor to pack."""
    rows, width = x.shape
    n = ops.ckpt8_bytes(rows, width)
    buf = torch.full((n + 32,), 0x5A, dtype=torch.uint8, device="cuda")
    ops.ckpt8_pack(t, out=buf[:n])
    codes, scales = _split(buf[:n], rows, width)
    want_codes, want_scales = R.pack_ref(x)
    assert torch.equal(scales, want_scales)
    # a NaN's sign and payload are free
    nan, want_nan = (codes & 127) == 127, (want_codes & 127) == 127
    assert torch.equal(nan, want_nan)
    assert torch.equal(codes[~nan], want_codes[~nan])
    assert bool((buf[n:] == 0x5A).all())
    return buf[:n], R.unpack_ref(codes, scales, width)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,width,pad", [(1, 1, 0), (1, 31, 0), (3, 32, 1), (5, 33, 0), (2, 64, 8),
                                            (17, 515, 3), (4, 2048, 0), (300, 96, 5), (1, 5120, 0)])
def test_pack_and_unpack(io, rows, width, pad):
    dtype = R.DTYPES[io]
    x = R.draw(rows * 1000 + width, rows, width, limit=50.0) * torch.logspace(-4, 4, width)
    x = x.to(dtype)
    ck, want = _check(x, R.strided(x.float(), pad, dtype))
    for to in ("f32", "bf16"):
        out = R.strided(torch.zeros(rows, width), pad, R.DTYPES[to])
        ops.ckpt8_unpack(ck, rows, width, out=out)
        assert torch.equal(out.cpu().double(), want)  # code * 2^k fits both types
        assert R.padding_untouched(out)
    assert ops.ckpt8_unpack(ck, rows, width, io="f32").dtype == torch.float32


def test_ties_and_borders():
    """Every bf16 value of two octaves (ties of the e4m3 grid among them), and
    blocks whose largest value sits at and next to 448 * 2^k."""
    x = torch.zeros(40, 64)
    m = torch.arange(256).float() / 128 + 1
    x[:8, :32] = m[:256].view(8, 32)
    x[:8, 32:] = -m.view(8, 32) * 2.0 ** -9  # down into the subnormal codes
    x[:, 31] = 448.0
    for i in range(8, 40):
        k = 2.0 ** (i - 24)
        x[i, :32] = 448.0 * k * torch.linspace(-1, 1, 32)
        x[i, 32:] = 449.0 * k * torch.linspace(-1, 1, 32)
    _check(x, x.cuda())
    _check(x.bfloat16(), x.bfloat16().cuda())


def test_extremes():
    tiny, big = torch.finfo(torch.float32).tiny, torch.finfo(torch.float32).max
    x = torch.zeros(6, 96)
    x[0] = torch.linspace(-1, 1, 96) * big
    x[1] = torch.linspace(-1, 1, 96) * tiny
    x[2] = torch.linspace(-1, 1, 96) * tiny * 2.0 ** -10   # subnormal inputs
    x[3, ::2] = -0.0
    x[4, 0], x[4, 40], x[4, 41], x[4, 95] = big, tiny, 1.0, float("nan")
    x[5] = float("inf")
    x[5, 32:64] = torch.linspace(1, 2, 32)
    x[5, 40], x[5, 41] = float("nan"), -float("inf")
    ck, want = _check(x, x.cuda())
    back = ops.ckpt8_unpack(ck, 6, 96, io="f32").cpu().double()
    assert torch.equal(torch.isnan(back), torch.isnan(want))
    assert torch.equal(back[~torch.isnan(want)], want[~torch.isnan(want)])


def test_no_rows():
    x = torch.zeros(0, 64, device="cuda")
    ck = ops.ckpt8_pack(x)
    assert ck.numel() == 0 and ops.ckpt8_unpack(ck, 0, 64).shape == (0, 64)


def test_far_rows():
    """Rows past 2^32 elements of a wide matrix, as a slice of it."""
    rows, width, ld = 70000, 40, 65536
    wide = torch.empty(rows, ld, dtype=torch.bfloat16, device="cuda")
    t = wide[:, 100:100 + width]
    x = R.draw(5, rows, width).bfloat16()
    t.copy_(x)
    ck = ops.ckpt8_pack(t)
    codes, scales = _split(ck, rows, width)
    sel = torch.tensor([0, 1, 32767, 32768, 65535, 65536, 69999])
    want_codes, want_scales = R.pack_ref(x[sel])
    assert torch.equal(codes[sel], want_codes) and torch.equal(scales[sel], want_scales)
    back = ops.ckpt8_unpack(ck, rows, width, out=wide[:, 7:7 + width])
    assert torch.equal(back[sel].cpu().double(), R.unpack_ref(want_codes, want_scales, width))
