"""The gated norm after the scan on the GPU against tests/block_ref.py in
float64: both gate orders, groups, widths of every kernel shape and odd ones,
row strides, f32 and bf16, the backward from tensors and from 8-bit
checkpoints."""
import pytest
import torch

import block_ref as R
import selective_scan_recurrence_amd as ssm
from selective_scan_recurrence_amd import ops

pytestmark = pytest.mark.gpu

EPS = 1e-5
# rows, width, groups, pad: a unit of 8, 16, 32, 64 lanes, a wave with two
# pieces, a workgroup with 1, 2, 4 pieces; exact and ragged ends
SHAPES = [(1, 1, 1, 0), (3, 8, 1, 1), (70, 61, 1, 0), (33, 64, 1, 8), (9, 128, 1, 0), (5, 250, 1, 3),
          (40, 512, 2, 0), (6, 500, 1, 12), (7, 1000, 1, 5), (5, 1024, 1, 0), (4, 2560, 1, 16),
          (3, 5120, 8, 0), (6, 771, 3, 1), (2, 8190, 1, 0), (2, 9000, 1, 2), (1, 32768, 1, 0),
          (2, 16640, 1, 8), (130, 96, 3, 0)]


def _inputs(rows, width, pad, io, gate=True, seed=0):
    dt = R.DTYPES[io]
    y = (R.draw(seed + 1, rows, width) * 1.5).to(dt)
    z = R.draw(seed + 2, rows, width, std=2.0).to(dt) if gate else None
    w = 1 + 0.2 * R.draw(seed + 3, width)
    return y, z, w, (None if z is None else R.strided(z.float(), pad, dt))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("after", [False, True])
@pytest.mark.parametrize("rows,width,groups,pad", SHAPES)
def test_forward_and_backward(rows, width, groups, pad, after, io):
    dt = R.DTYPES[io]
    y, z, w, zd = _inputs(rows, width, pad, io, seed=width)
    d = ops.norm_desc(n_rows=rows, width=width, n_group=groups, io=io, eps=EPS, gate_after=after,
                      ld_z=width + pad, ld_out=width + pad)
    out = R.strided(torch.zeros(rows, width), pad, dt)
    rstd = torch.empty(rows, groups, device="cuda")
    ops.norm_gated_fwd(d, y.cuda(), zd, w.cuda(), out=out, rstd=rstd)
    want, inv = R.gated_fwd(y.double(), z.double(), w.double(), groups, EPS, after)
    R.check("out", out, want, want.abs(), io)
    R.check("rstd", rstd, inv, inv, "f32")
    assert R.padding_untouched(out)
    dout = R.draw(width + 9, rows, width).to(dt)
    g = ops.norm_gated_bwd(d, R.strided(dout.float(), pad, dt), w.cuda(), rstd, y=y.cuda(), z=zd,
                           d_z=R.strided(torch.zeros(rows, width), pad, dt))
    want = R.gated_bwd(dout.double(), y.double(), z.double(), w.double(), inv, groups, after)
    R.check("d_y", g.d_y, *want["d_y"], io)
    R.check("d_z", g.d_z, *want["d_z"], io)
    R.check("d_w", g.d_w, *want["d_w"], "f32", R.COUNT_SUM)
    assert R.padding_untouched(g.d_z)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,width,groups", [(5, 2880, 4), (3, 4160, 4), (4, 2880, 40), (300, 72, 3),
                                               (2, 8192, 1024), (7, 1344, 7)])
def test_many_groups(rows, width, groups, io):
    """Groups whose sums span lanes and waves of a row, one piece each, more
    groups than waves."""
    dt = R.DTYPES[io]
    y, z, w, zd = _inputs(rows, width, 0, io, seed=width)
    d = ops.norm_desc(n_rows=rows, width=width, n_group=groups, io=io, eps=EPS)
    rstd = torch.empty(rows, groups, device="cuda")
    r = ops.norm_gated_fwd(d, y.cuda(), zd, w.cuda(), rstd=rstd)
    want, inv = R.gated_fwd(y.double(), z.double(), w.double(), groups, EPS)
    R.check("out", r.out, want, want.abs(), io)
    R.check("rstd", rstd, inv, inv, "f32")
    dout = R.draw(width + 9, rows, width).to(dt)
    g = ops.norm_gated_bwd(d, dout.cuda(), w.cuda(), rstd, y=y.cuda(), z=zd)
    want = R.gated_bwd(dout.double(), y.double(), z.double(), w.double(), inv, groups)
    R.check("d_y", g.d_y, *want["d_y"], io)
    R.check("d_z", g.d_z, *want["d_z"], io)
    R.check("d_w", g.d_w, *want["d_w"], "f32", R.COUNT_SUM)


@pytest.mark.parametrize("rows,width,groups,after,io", [(32768, 523, 1, False, "bf16"), (33001, 640, 1, True, "bf16"),
                                                        (32771, 1042, 2, False, "bf16"), (32769, 1024, 1, False, "f32"),
                                                        (32767, 768, 1, False, "bf16")])
def test_many_rows_of_middling_width(rows, width, groups, after, io):
    """Groups of 520 to 1024 columns in both forms, of few rows and of many.  A
    sum over the rows adds at most 17 of them in a lane, then up to 64 partial
    rows in each of 32 lanes, and those."""
    dt = R.DTYPES[io]
    y, z, w, zd = _inputs(rows, width, 0, io, seed=width)
    d = ops.norm_desc(n_rows=rows, width=width, n_group=groups, io=io, eps=EPS, gate_after=after)
    rstd = torch.empty(rows, groups, device="cuda")
    ops.norm_gated_fwd(d, y.cuda(), zd, w.cuda(), rstd=rstd)
    _, inv = R.gated_fwd(y.double(), z.double(), w.double(), groups, EPS, after)
    dout = R.draw(width + 9, rows, width).to(dt)
    g = ops.norm_gated_bwd(d, dout.cuda(), w.cuda(), rstd, y=y.cuda(), z=zd)
    want = R.gated_bwd(dout.double(), y.double(), z.double(), w.double(), inv, groups, after)
    R.check("d_y", g.d_y, *want["d_y"], io)
    R.check("d_z", g.d_z, *want["d_z"], io)
    R.check("d_w", g.d_w, *want["d_w"], "f32", R.COUNT + 17 + 64 + 32)


@pytest.mark.parametrize("after", [False, True])
@pytest.mark.parametrize("rows,width,groups", [(12000, 5120, 8), (24000, 2048, 1), (400000, 128, 1)])
def test_matrices_past_the_cache(rows, width, groups, after):
    """Calls large enough to store past the caches give, row by row, what a
    call on a few of their rows gives."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    y, z, dout = (torch.randn(rows, width, generator=gen, device="cuda").bfloat16() for _ in range(3))
    w = torch.rand(width, generator=gen, device="cuda") + 0.5

    def run(y, z, dout):
        d = ops.norm_desc(n_rows=y.shape[0], width=width, n_group=groups, eps=EPS, gate_after=after)
        f = ops.norm_gated_fwd(d, y, z, w, train=True)
        g = ops.norm_gated_bwd(d, dout, w, f.rstd, y=y, z=z)
        return f.out, f.rstd, g.d_y, g.d_z

    some = torch.cat([torch.arange(5), torch.arange(rows // 2, rows // 2 + 40), torch.arange(rows - 6, rows)]).cuda()
    for big, small in zip(run(y, z, dout), run(y[some], z[some], dout[some])):
        assert torch.equal(big[some], small)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("after", [False, True])
@pytest.mark.parametrize("rows,width,groups", [(5, 64, 1), (33, 256, 8), (7, 515, 1), (4, 5120, 8),
                                               (3, 10240, 1), (300, 40, 1)])
def test_backward_from_checkpoints(rows, width, groups, after, io):
    dt = R.DTYPES[io]
    y, z, w, zd = _inputs(rows, width, 0, io, seed=width + 1)
    d = ops.norm_desc(n_rows=rows, width=width, n_group=groups, io=io, eps=EPS, gate_after=after)
    yd = y.cuda()
    r = ops.norm_gated_fwd(d, yd, zd, w.cuda(), train=True, out8=ops.ckpt8_empty(rows, width))
    # what the fused checkpoints hold is what packing the tensors holds
    assert torch.equal(r.y8, ops.ckpt8_pack(yd))
    assert torch.equal(r.z8, ops.ckpt8_pack(zd))
    assert torch.equal(r.out8, ops.ckpt8_pack(r.out))
    inv = R.gated_fwd(y.double(), z.double(), w.double(), groups, EPS, after)[1]
    dout = R.draw(width + 9, rows, width).to(dt)
    kept_y, kept_z = R.kept(y), R.kept(z)
    for case in ("both", "y", "z"):
        args = {"both": dict(y8=r.y8, z8=r.z8), "y": dict(y8=r.y8, z=zd), "z": dict(y=yd, z8=r.z8)}[case]
        g = ops.norm_gated_bwd(d, dout.cuda(), w.cuda(), r.rstd, **args)
        want = R.gated_bwd(dout.double(), kept_y if "y8" in args else y.double(),
                           kept_z if "z8" in args else z.double(), w.double(), inv, groups, after)
        R.check("d_y", g.d_y, *want["d_y"], io)
        R.check("d_z", g.d_z, *want["d_z"], io)
        R.check("d_w", g.d_w, *want["d_w"], "f32", R.COUNT_SUM)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_without_gate(io):
    rows, width, dt = 19, 300, R.DTYPES[io]
    y, _, w, _ = _inputs(rows, width, 0, io, gate=False)
    d = ops.norm_desc(n_rows=rows, width=width, io=io, eps=EPS)
    r = ops.norm_gated_fwd(d, y.cuda(), None, w.cuda(), train=True)
    want, inv = R.gated_fwd(y.double(), None, w.double(), 1, EPS)
    R.check("out", r.out, want, want.abs(), io)
    assert r.z8 is None
    dout = R.draw(3, rows, width).to(dt)
    g = ops.norm_gated_bwd(d, dout.cuda(), w.cuda(), r.rstd, y=y.cuda())
    want = R.gated_bwd(dout.double(), y.double(), None, w.double(), inv)
    R.check("d_y", g.d_y, *want["d_y"], io)
    R.check("d_w", g.d_w, *want["d_w"], "f32", R.COUNT_SUM)
    assert g.d_z is None


@pytest.mark.parametrize("rows", [0, 1, 2, 1777, 4096])
def test_row_counts(rows):
    """No rows (d_w is then zero) up to many, where workgroups share them."""
    width = 72
    y, z, w, zd = _inputs(max(rows, 1), width, 0, "bf16")
    y, z, zd = y[:rows], z[:rows], zd[:rows]
    d = ops.norm_desc(n_rows=rows, width=width, eps=EPS)
    r = ops.norm_gated_fwd(d, y.cuda(), zd, w.cuda(), train=True)
    dout = R.draw(7, max(rows, 1), width).to(torch.bfloat16)[:rows]
    g = ops.norm_gated_bwd(d, dout.cuda(), w.cuda(), r.rstd, y=y.cuda(), z=zd,
                           d_w=torch.full((width,), float("nan"), device="cuda"))
    if rows == 0:
        assert not g.d_w.any()
        return
    want, inv = R.gated_fwd(y.double(), z.double(), w.double(), 1, EPS)
    R.check("out", r.out, want, want.abs(), "bf16")
    want = R.gated_bwd(dout.double(), y.double(), z.double(), w.double(), inv)
    R.check("d_y", g.d_y, *want["d_y"], "bf16")
    R.check("d_w", g.d_w, *want["d_w"], "f32", R.COUNT_SUM)


def test_zero_and_nan_rows():
    """A row of zeros has rstd = eps^-1/2 and zero output; a NaN or an infinity
    stays in its row, and in d_w."""
    y, z, w, zd = _inputs(6, 130, 0, "f32")
    y[1] = 0.0
    y[3, 77], y[4, 0] = float("nan"), float("inf")
    d = ops.norm_desc(n_rows=6, width=130, io="f32", eps=EPS)
    r = ops.norm_gated_fwd(d, y.cuda(), zd, w.cuda(), train=True)
    out = r.out.cpu()
    assert not out[1].any() and abs(float(r.rstd[1]) * EPS ** 0.5 - 1) < 1e-6
    assert torch.isnan(out[3]).all() and torch.isnan(out[4, 0])
    good = [0, 2, 5]
    want = R.gated_fwd(y[good].double(), z[good].double(), w.double(), 1, EPS)[0]
    R.check("out", r.out[good], want, want.abs(), "f32")
    g = ops.norm_gated_bwd(d, torch.ones(6, 130, device="cuda"), w.cuda(), r.rstd, y8=r.y8, z8=r.z8)
    assert torch.isfinite(g.d_y[[0, 1, 2, 5]]).all() and torch.isnan(g.d_y[3]).all()
    assert torch.isnan(g.d_w[77])


def test_large_gates():
    """Gates far outside e^-z's range: SiLU is 0 or z itself, without NaN."""
    y, _, w, _ = _inputs(2, 64, 0, "f32")
    z = torch.linspace(-200, 200, 128).view(2, 64)
    d = ops.norm_desc(n_rows=2, width=64, io="f32", eps=EPS)
    r = ops.norm_gated_fwd(d, y.cuda(), z.cuda(), w.cuda(), train=True)
    g = ops.norm_gated_bwd(d, y.cuda(), w.cuda(), r.rstd, y=y.cuda(), z=z.cuda())
    for t in (r.out, g.d_y, g.d_z, g.d_w):
        assert torch.isfinite(t).all()


def test_repeats_bitwise():
    y, z, w, zd = _inputs(2000, 640, 0, "bf16")
    d = ops.norm_desc(n_rows=2000, width=640, n_group=2, eps=EPS)
    yd, wd, dout = y.cuda(), w.cuda(), R.draw(5, 2000, 640).bfloat16().cuda()
    runs = []
    for _ in range(3):
        r = ops.norm_gated_fwd(d, yd, zd, wd, train=True)
        runs.append((r, ops.norm_gated_bwd(d, dout, wd, r.rstd, y8=r.y8, z8=r.z8)))
    for r, g in runs[1:]:
        assert torch.equal(r.out, runs[0][0].out) and torch.equal(r.rstd, runs[0][0].rstd)
        for k in ("d_y", "d_z", "d_w"):
            assert torch.equal(getattr(g, k), getattr(runs[0][1], k))


def test_refused_on_the_device():
    d = ops.norm_desc(n_rows=4, width=96, n_group=2)
    y = torch.zeros(4, 96, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(96, device="cuda")
    for bad in (dict(train=True), dict(out=y[:, :64]), dict(rstd=w[:7])):
        with pytest.raises(ssm.SsmError):
            ops.norm_gated_fwd(d, y, y, w, **bad)


def test_far_rows():
    """z as a slice whose rows lie past 2^32 elements."""
    rows, width, ld = 70000, 24, 65536
    wide = torch.empty(rows, ld, dtype=torch.bfloat16, device="cuda")
    zd = wide[:, 50:50 + width]
    z, y = R.draw(1, rows, width).bfloat16(), R.draw(2, rows, width).bfloat16()
    zd.copy_(z)
    w = 1 + 0.1 * R.draw(3, width)
    d = ops.norm_desc(n_rows=rows, width=width, ld_z=ld, eps=EPS)
    r = ops.norm_gated_fwd(d, y.cuda(), zd, w.cuda(), train=True)
    want, inv = R.gated_fwd(y.double(), z.double(), w.double(), 1, EPS)
    R.check("out", r.out, want, want.abs(), "bf16")
    dout = R.draw(4, rows, width).bfloat16()
    g = ops.norm_gated_bwd(d, dout.cuda(), w.cuda(), r.rstd, y=y.cuda(), z=zd, d_z=zd)
    want = R.gated_bwd(dout.double(), y.double(), z.double(), w.double(), inv)
    R.check("d_z", zd, *want["d_z"], "bf16")
    R.check("d_y", g.d_y, *want["d_y"], "bf16")
