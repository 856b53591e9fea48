"""The norm between two blocks on the GPU against tests/block_ref.py in
float64: with and without the norm after the block and the learned scale,
every kernel shape, row strides, the stream in f32 and bf16 and in place, the
backward from tensors and from 8-bit checkpoints."""
import pytest
import torch

import block_ref as R
import selective_scan_recurrence_amd as ssm
from selective_scan_recurrence_amd import ops

pytestmark = pytest.mark.gpu

EPS = 1e-5
TYPES = [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")]
SHAPES = [(1, 1, 0), (3, 8, 1), (70, 61, 0), (33, 64, 8), (9, 128, 0), (5, 250, 3), (40, 256, 0),
          (6, 500, 12), (7, 1000, 5), (5, 1024, 0), (9, 768, 0), (11, 523, 1), (4, 2560, 16), (2, 8190, 0), (2, 9000, 2),
          (1, 32768, 0), (2, 16640, 8)]


def _inputs(rows, width, io, res, post, scale, seed=0):
    b = (R.draw(seed + 1, rows, width) * 2).to(R.DTYPES[io])
    r = (R.draw(seed + 2, rows, width) * 3).to(R.DTYPES[res])
    w, wp, sc = (1 + 0.2 * R.draw(seed + k, width) for k in (3, 4, 5))
    return b, r, w, wp if post else None, 0.3 * sc if scale else None


def _d(t):
    return None if t is None else t.double()


def _c(t):
    return None if t is None else t.cuda()


def _check_grads(g, want, io, res):
    R.check("d_r", g.d_r, *want["d_r"], res)
    R.check("d_b", g.d_b, *want["d_b"], io)
    for k in ("d_w", "d_w_post", "d_scale"):
        if k in want:
            R.check(k, getattr(g, k), *want[k], "f32", R.COUNT_SUM)
        else:
            assert getattr(g, k) is None


@pytest.mark.parametrize("io,res", TYPES)
@pytest.mark.parametrize("post,scale", [(False, False), (True, True), (True, False), (False, True)])
@pytest.mark.parametrize("rows,width,pad", SHAPES)
def test_forward_and_backward(rows, width, pad, post, scale, io, res):
    b, r, w, wp, sc = _inputs(rows, width, io, res, post, scale, seed=width)
    dio, dres, ld = R.DTYPES[io], R.DTYPES[res], width + pad
    d = ops.norm_desc(n_rows=rows, width=width, io=io, res=res, eps=EPS, res_scale=0.7, ld_x=ld,
                      ld_res=ld, ld_out=ld)
    bd, rd = R.strided(b.float(), pad, dio), R.strided(r.float(), pad, dres)
    r_out, h = (R.strided(torch.zeros(rows, width), pad, t) for t in (dres, dio))
    rstd = torch.empty(rows, device="cuda")
    rstd_post = torch.empty(rows, device="cuda") if post else None
    ops.norm_residual_fwd(d, bd, rd, w.cuda(), w_post=_c(wp), scale=_c(sc), r_out=r_out, h=h,
                          rstd=rstd, rstd_post=rstd_post)
    x, want_h, inv, inv_post, mag = R.residual_fwd(b.double(), r.double(), w.double(), _d(wp), _d(sc),
                                                   0.7, EPS)
    R.check("r_out", r_out, x, mag, res)
    R.check("h", h, want_h, mag * inv.unsqueeze(-1) * w.double().abs() + want_h.abs(), io)
    R.check("rstd", rstd, inv, inv * (1 + (mag * x.abs()).mean(-1) * inv ** 2), "f32")
    if post:
        R.check("rstd_post", rstd_post, inv_post, inv_post, "f32")
    assert R.padding_untouched(r_out) and R.padding_untouched(h)
    # the gradient at the stored stream
    dh, dr = R.draw(width + 8, rows, width).to(dio), R.draw(width + 9, rows, width).to(dres)
    stored = r_out.double().cpu()
    g = ops.norm_residual_bwd(d, R.strided(dh.float(), pad, dio), w.cuda(), rstd,
                              dr_out=R.strided(dr.float(), pad, dres), r_out=r_out,
                              b=bd if post or scale else None, rstd_post=rstd_post, w_post=_c(wp),
                              scale=_c(sc), d_r=R.strided(torch.zeros(rows, width), pad, dres),
                              d_b=R.strided(torch.zeros(rows, width), pad, dio))
    want = R.residual_bwd(dh.double(), dr.double(), stored, b.double(), w.double(), rstd.double().cpu(),
                          _d(rstd_post.cpu()) if post else None, _d(wp), _d(sc), 0.7)
    _check_grads(g, want, io, res)
    assert R.padding_untouched(g.d_r) and R.padding_untouched(g.d_b)


@pytest.mark.parametrize("io,res", TYPES)
@pytest.mark.parametrize("post,scale", [(False, False), (True, True), (False, True)])
@pytest.mark.parametrize("rows,width", [(5, 64), (33, 200), (7, 515), (4, 2560), (2, 10240), (300, 40)])
def test_backward_from_checkpoints(rows, width, post, scale, io, res):
    b, r, w, wp, sc = _inputs(rows, width, io, res, post, scale, seed=width + 1)
    d = ops.norm_desc(n_rows=rows, width=width, io=io, res=res, eps=EPS, res_scale=0.5)
    bd = b.cuda()
    f = ops.norm_residual_fwd(d, bd, r.cuda(), w.cuda(), w_post=_c(wp), scale=_c(sc), train=True)
    # what the fused checkpoints hold is what packing the stored tensors holds
    assert torch.equal(f.r8, ops.ckpt8_pack(f.r_out))
    assert torch.equal(f.h8, ops.ckpt8_pack(f.h))
    assert (f.b8 is not None) == (post or scale)
    if f.b8 is not None:
        assert torch.equal(f.b8, ops.ckpt8_pack(bd))
    dh, dr = R.draw(8, rows, width).to(R.DTYPES[io]), R.draw(9, rows, width).to(R.DTYPES[res])
    g = ops.norm_residual_bwd(d, dh.cuda(), w.cuda(), f.rstd, dr_out=dr.cuda(), r8=f.r8, b8=f.b8,
                              rstd_post=f.rstd_post, w_post=_c(wp), scale=_c(sc))
    want = R.residual_bwd(dh.double(), dr.double(), R.kept(f.r_out.cpu()), R.kept(b), w.double(),
                          f.rstd.double().cpu(), _d(f.rstd_post.cpu()) if post else None, _d(wp), _d(sc),
                          0.5)
    _check_grads(g, want, io, res)


@pytest.mark.parametrize("missing", ["b", "r", "dr_out"])
def test_optional_inputs(missing):
    rows, width = 21, 130
    b, r, w, _, _ = _inputs(rows, width, "bf16", "f32", False, False)
    d = ops.norm_desc(n_rows=rows, width=width, eps=EPS)
    zero = torch.zeros(rows, width)
    f = ops.norm_residual_fwd(d, None if missing == "b" else b.cuda(), None if missing == "r" else r.cuda(),
                              w.cuda(), train=True)
    x, h, inv, _, mag = R.residual_fwd((zero if missing == "b" else b).double(),
                                       (zero if missing == "r" else r).double(), w.double(), eps=EPS)
    R.check("r_out", f.r_out, x, mag, "f32")
    R.check("h", f.h, h, mag * inv.unsqueeze(-1) * w.double() + h.abs(), "bf16")
    dh, dr = R.draw(8, rows, width).bfloat16(), R.draw(9, rows, width)
    g = ops.norm_residual_bwd(d, dh.cuda(), w.cuda(), f.rstd, r_out=f.r_out,
                              dr_out=None if missing == "dr_out" else dr.cuda())
    want = R.residual_bwd(dh.double(), (zero if missing == "dr_out" else dr).double(),
                          f.r_out.double().cpu(), b.double(), w.double(), f.rstd.double().cpu())
    _check_grads(g, want, "bf16", "f32")


@pytest.mark.parametrize("width", [60, 700, 2560, 20000])
def test_in_place(width):
    """r_out = r and d_r = dr_out give what separate tensors give."""
    rows = 50
    b, r, w, wp, sc = _inputs(rows, width, "bf16", "f32", True, True)
    d = ops.norm_desc(n_rows=rows, width=width, eps=EPS)
    kw = dict(w_post=wp.cuda(), scale=sc.cuda())
    f = ops.norm_residual_fwd(d, b.cuda(), r.cuda(), w.cuda(), train=True, **kw)
    stream = r.cuda()
    f2 = ops.norm_residual_fwd(d, b.cuda(), stream, w.cuda(), train=True, r_out=stream, **kw)
    assert torch.equal(stream, f.r_out) and torch.equal(f2.h, f.h)
    dh, dr = R.draw(8, rows, width).bfloat16().cuda(), R.draw(9, rows, width).cuda()
    args = dict(r8=f.r8, b8=f.b8, rstd_post=f.rstd_post, **kw)
    g = ops.norm_residual_bwd(d, dh, w.cuda(), f.rstd, dr_out=dr, **args)
    g2 = ops.norm_residual_bwd(d, dh, w.cuda(), f.rstd, dr_out=dr, d_r=dr, **args)
    assert torch.equal(dr, g.d_r) and torch.equal(g2.d_b, g.d_b) and torch.equal(g2.d_scale, g.d_scale)


@pytest.mark.parametrize("rows", [0, 1, 1777, 4096])
def test_row_counts(rows):
    width = 72
    b, r, w, wp, sc = _inputs(max(rows, 1), width, "bf16", "f32", True, True)
    b, r = b[:rows], r[:rows]
    d = ops.norm_desc(n_rows=rows, width=width, eps=EPS)
    kw = dict(w_post=wp.cuda(), scale=sc.cuda())
    f = ops.norm_residual_fwd(d, b.cuda(), r.cuda(), w.cuda(), train=True, **kw)
    dh, dr = (R.draw(k, max(rows, 1), width)[:rows] for k in (8, 9))
    dh = dh.bfloat16()
    nan = torch.full((3, width), float("nan"), device="cuda")
    g = ops.norm_residual_bwd(d, dh.cuda(), w.cuda(), f.rstd, dr_out=dr.cuda(), r_out=f.r_out, b=b.cuda(),
                              rstd_post=f.rstd_post, d_w=nan[0], d_w_post=nan[1], d_scale=nan[2], **kw)
    if rows == 0:
        assert not nan.any()
        return
    want = R.residual_bwd(dh.double(), dr.double(), f.r_out.double().cpu(), b.double(), w.double(),
                          f.rstd.double().cpu(), f.rstd_post.double().cpu(), wp.double(), sc.double())
    _check_grads(g, want, "bf16", "f32")


def test_zero_and_nan_rows():
    b, r, w, _, _ = _inputs(5, 90, "f32", "f32", False, False)
    b[1] = r[1] = 0.0
    r[3, 40] = float("nan")
    d = ops.norm_desc(n_rows=5, width=90, io="f32", eps=EPS)
    f = ops.norm_residual_fwd(d, b.cuda(), r.cuda(), w.cuda(), train=True)
    assert not f.h[1].any() and torch.isnan(f.h[3]).all()
    assert torch.isfinite(f.r_out[3]).sum() == 89
    assert torch.isfinite(f.h[[0, 2, 4]]).all()
    g = ops.norm_residual_bwd(d, b.cuda(), w.cuda(), f.rstd, r8=f.r8)
    assert torch.isfinite(g.d_r[[0, 1, 2, 4]]).all() and torch.isnan(g.d_w[40])


def test_gradients_asked_one_by_one():
    """Each output may be left out; the others do not change."""
    rows, width = 37, 300
    b, r, w, wp, sc = _inputs(rows, width, "bf16", "f32", True, True)
    d = ops.norm_desc(n_rows=rows, width=width, eps=EPS)
    f = ops.norm_residual_fwd(d, b.cuda(), r.cuda(), w.cuda(), train=True, w_post=wp.cuda(), scale=sc.cuda())
    dh, dr = R.draw(8, rows, width).bfloat16().cuda(), R.draw(9, rows, width).cuda()
    wd, wpd, scd = w.cuda(), wp.cuda(), sc.cuda()
    ws = ops.norm_bwd_workspace(d)
    full = ops.norm_residual_bwd(d, dh, wd, f.rstd, dr_out=dr, r8=f.r8, b8=f.b8, rstd_post=f.rstd_post,
                                 w_post=wpd, scale=scd)
    names = ["d_r", "d_b", "d_w", "d_w_post", "d_scale"]
    for k in range(5):
        outs = [torch.empty_like(getattr(full, n)) if i == k else None for i, n in enumerate(names)]
        ssm.ssm_norm_residual_bwd(d, dh, dr, None, f.r8, None, f.b8, wpd, scd, wd, f.rstd, f.rstd_post,
                                  *outs, ws, ws.numel())
        assert torch.equal(outs[k], getattr(full, names[k])), names[k]


def test_repeats_bitwise():
    rows, width = 3000, 320
    b, r, w, wp, sc = _inputs(rows, width, "bf16", "f32", True, True)
    d = ops.norm_desc(n_rows=rows, width=width, eps=EPS)
    kw = dict(w_post=wp.cuda(), scale=sc.cuda())
    bd, rd, wd = b.cuda(), r.cuda(), w.cuda()
    dh, dr = R.draw(8, rows, width).bfloat16().cuda(), R.draw(9, rows, width).cuda()
    runs = []
    for _ in range(3):
        f = ops.norm_residual_fwd(d, bd, rd, wd, train=True, **kw)
        g = ops.norm_residual_bwd(d, dh, wd, f.rstd, dr_out=dr, r8=f.r8, b8=f.b8, rstd_post=f.rstd_post, **kw)
        runs.append([f.r_out, f.h, g.d_r, g.d_b, g.d_w, g.d_w_post, g.d_scale])
    for other in runs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(runs[0], other))
