"""The operators around the scan at the far ends of what they take."""
import pytest
import torch

import block_ref as R
from selective_scan_recurrence_amd import ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_wgrad_of_the_most_rows(io):
    """2147482623 rows, whose last part ends past 2^31 - 1 before it is cut to the
    rows: every part's rows count.  All zero but for ones, at the ends of the
    rows and along them, so that dw counts them."""
    rows, width, n_out = 2147482623, 32, 4
    dtype = torch.float32 if io == "f32" else torch.bfloat16
    need = ops.ckpt8_bytes(rows, width) + rows * n_out * dtype.itemsize
    if torch.cuda.mem_get_info()[0] < need + (4 << 30):
        pytest.skip("needs 110 GB of free device memory")
    at = torch.tensor([0, 1, 4194303, 4194304, 8388608, 1 << 30, 2143289343, 2143289344, 2143289345,
                       2147000000, rows - 65, rows - 64, rows - 1], device="cuda")
    ck = torch.zeros(ops.ckpt8_bytes(rows, width), dtype=torch.uint8, device="cuda")
    ck[:rows * width].view(rows, width)[at] = 0x38  # 1.0, with the scale 2^0
    ck[rows * width:][at] = 127
    dy = torch.zeros(rows, n_out, dtype=dtype, device="cuda")
    dy[at] = 1.0
    dw = ops.ckpt8_wgrad(dy, ck, width)
    torch.cuda.synchronize()
    del ck, dy
    torch.cuda.empty_cache()
    assert bool((dw == len(at)).all()), dw


# rows, width, groups: a unit of 4 to 64 lanes, a wave with two pieces, 32 lanes
# with three (residual), a workgroup with 1, 2, 4 pieces a lane, rows with all
# their groups in a workgroup; exact and ragged ends
ROWS = [(9, 24, 1), (70, 61, 1), (33, 64, 1), (40, 128, 1), (9, 250, 1), (40, 1024, 2), (7, 1000, 1), (6, 768, 1),
        (5, 2560, 1), (6, 771, 3), (9, 5120, 8), (300, 72, 3), (3, 2880, 40), (3, 9000, 1), (2, 16640, 1)]


def _huge(seed, rows, width, groups, dtype):
    """Rows of ordinary values, and a group in every second row whose finite
    values have squares that add up past the largest f32."""
    x = R.draw(seed, rows, width)
    for i in range(0, rows, 2):
        g = i // 2 % groups
        x[i, g * width // groups:(g + 1) * width // groups] *= 2.0 ** (63 + 12 * (i % 4))
    return x.to(dtype)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("after", [False, True])
@pytest.mark.parametrize("rows,width,groups", ROWS)
def test_gated_norm_of_huge_values(rows, width, groups, after, io):
    """Rows whose sum of squares passes f32 are normalised as any other, and
    leave their neighbours alone."""
    y = _huge(width, rows, width, groups, R.DTYPES[io])
    z, dout = (R.draw(width + k, rows, width).to(R.DTYPES[io]) for k in (1, 2))
    w = 1 + 0.2 * R.draw(width + 3, width)
    d = ops.norm_desc(n_rows=rows, width=width, n_group=groups, io=io, gate_after=after)
    rstd = torch.empty(rows, groups, device="cuda")
    f = ops.norm_gated_fwd(d, y.cuda(), z.cuda(), w.cuda(), rstd=rstd)
    want, inv = R.gated_fwd(y.double(), z.double(), w.double(), groups, 1e-5, after)
    R.check("out", f.out, want, want.abs(), io)
    R.check("rstd", rstd, inv, inv, "f32")
    g = ops.norm_gated_bwd(d, dout.cuda(), w.cuda(), rstd, y=y.cuda(), z=z.cuda())
    want = R.gated_bwd(dout.double(), y.double(), z.double(), w.double(), inv, groups, after)
    R.check("d_y", g.d_y, *want["d_y"], io)
    R.check("d_z", g.d_z, *want["d_z"], io)
    R.check("d_w", g.d_w, *want["d_w"], "f32", R.COUNT_SUM)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("huge", ["b", "r"])
@pytest.mark.parametrize("rows,width", [(m, n) for m, n, g in ROWS if g == 1])
def test_residual_norm_of_huge_values(rows, width, huge, io):
    """The same for both sums of the residual norm: of the branch, and of the stream."""
    b, r = R.draw(width, rows, width).to(R.DTYPES[io]), R.draw(width + 1, rows, width)
    if huge == "b":
        b = _huge(width, rows, width, 1, R.DTYPES[io])
    else:
        r = _huge(width + 1, rows, width, 1, torch.float32)
    w, wp = (1 + 0.2 * R.draw(width + k, width) for k in (2, 3))
    d = ops.norm_desc(n_rows=rows, width=width, io=io, res_scale=0.7)
    rstd, post = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    f = ops.norm_residual_fwd(d, b.cuda(), r.cuda(), w.cuda(), w_post=wp.cuda(), rstd=rstd, rstd_post=post)
    x, h, inv, inv_post, mag = R.residual_fwd(b.double(), r.double(), w.double(), wp.double(), None, 0.7)
    R.check("r_out", f.r_out, x, mag, "f32")
    R.check("h", f.h, h, mag * inv.unsqueeze(-1) * w.double().abs() + h.abs(), io)
    R.check("rstd", rstd, inv, inv * (1 + (mag * x.abs()).mean(-1) * inv ** 2), "f32")
    R.check("rstd_post", post, inv_post, inv_post, "f32")


def test_infinities_keep_to_their_row():
    """A row that holds an infinity has rstd = 0; the rows beside it in a wave,
    huge or not, are as without it."""
    y, w = _huge(5, 8, 61, 1, torch.float32).cuda(), torch.ones(61, device="cuda")
    d = ops.norm_desc(n_rows=8, width=61, io="f32")
    rstd, rstd2 = torch.empty(8, 1, device="cuda"), torch.empty(8, 1, device="cuda")
    want = ops.norm_gated_fwd(d, y, None, w, rstd=rstd).out.clone()
    y[2, 60], y[5, 0], y[6, 7] = float("inf"), float("-inf"), float("nan")
    got = ops.norm_gated_fwd(d, y, None, w, rstd=rstd2).out
    ok = [0, 1, 3, 4, 7]
    assert torch.equal(got[ok], want[ok]) and torch.equal(rstd2[ok], rstd[ok])
    assert torch.isfinite(want).all() and bool(want.any(1).all())
    assert float(rstd2[2]) == 0.0 and float(rstd2[5]) == 0.0 and torch.isnan(rstd2[6]).all()
    assert torch.isnan(got[2, 60]) and not got[2, :60].any() and torch.isnan(got[6]).all()


@pytest.mark.parametrize("width", [20, 200, 900, 2560, 9000, 32768])
def test_norms_of_the_largest_values(width):
    """Rows of plus and minus the largest f32 have rms of that size and come out
    as plus and minus w.  (rstd = 2.9e-39 is subnormal, with steps of 2^-149:
    half of one is 2^-22 of it, which is 4 more half steps.)"""
    rows, top = 5, torch.finfo(torch.float32).max
    sign = torch.where(R.draw(width, rows, width) < 0, -1.0, 1.0)
    w = 1 + 0.2 * R.draw(width + 1, width)
    d = ops.norm_desc(n_rows=rows, width=width, io="f32")
    x = (sign * top).cuda()
    want = sign.double() * w.double()
    R.check("gated", ops.norm_gated_fwd(d, x, None, w.cuda()).out, want, want.abs(), "f32", R.COUNT + 4)
    R.check("residual", ops.norm_residual_fwd(d, None, x, w.cuda()).h, want, want.abs(), "f32", R.COUNT + 4)
