"""Unusual but possible arguments of the operators around the scan, on the GPU:
refused before a launch, or taken as they are meant."""
import pytest
import torch

import block_ref as R
import selective_scan_recurrence_amd as ssm
from selective_scan_recurrence_amd import ops

pytestmark = pytest.mark.gpu


def _status(f, *a, **kw):
    with pytest.raises(ssm.SsmError) as e:
        f(*a, **kw)
    return e.value.status


def test_expanded_rows():
    """The gradient of a sum over tokens is one row for all: refused as it is,
    taken once it is dense."""
    rows, width, n_out = 70, 96, 40
    g = R.draw(1, 1, n_out).bfloat16()
    x = R.draw(2, rows, width)
    ck = ops.ckpt8_pack(x.cuda())
    spread = g.cuda().expand(rows, n_out)
    assert _status(ops.ckpt8_wgrad, spread, ck, width) == ssm.SSM_ERR_SHAPE
    assert _status(ops.ckpt8_pack, spread) == ssm.SSM_ERR_SHAPE
    assert _status(ops.ckpt8_unpack, ck, rows, width,
                   out=torch.zeros(1, width, device="cuda").expand(rows, width)) == ssm.SSM_ERR_SHAPE
    got = ops.ckpt8_wgrad(spread.contiguous(), ck, width)
    dy, kept = g.double().expand(rows, n_out), R.kept(x)
    R.check("dw", got, dy.t() @ kept, dy.abs().t() @ kept.abs(), "f32", rows + 40)


def test_descriptor_without_strides():
    """Strides left 0 in the descriptor stand for dense rows."""
    rows, width = 9, 200
    y, z, d = (R.draw(k, rows, width).bfloat16().cuda() for k in (1, 2, 3))
    r, w = R.draw(4, rows, width).cuda(), (1 + 0.1 * R.draw(5, width)).cuda()
    raw = ssm.SsmNormDesc(rows, width, 1, 0, 0, 0, 0, ssm.SSM_BF16, ssm.SSM_F32, 1e-5, 1.0, 0, 0)
    runs = []
    for desc in (raw, ops.norm_desc(n_rows=rows, width=width)):
        f = ops.norm_gated_fwd(desc, y, z, w, train=True)
        g = ops.norm_gated_bwd(desc, d, w, f.rstd, y8=f.y8, z8=f.z8)
        n = ops.norm_residual_fwd(desc, y, r, w, train=True)
        m = ops.norm_residual_bwd(desc, d, w, n.rstd, r8=n.r8)
        runs.append([f.out, g.d_y, g.d_z, g.d_w, n.r_out, n.h, m.d_r, m.d_b, m.d_w])
    for a, b in zip(*runs):
        assert a.shape[-1] == width and torch.equal(a, b)


def test_workspace_in_host_memory():
    """A workspace that the GPU could not write is refused before the launch."""
    rows, width = 300, 96
    y, w = R.draw(1, rows, width).bfloat16().cuda(), torch.ones(width, device="cuda")
    d = ops.norm_desc(n_rows=rows, width=width)
    f = ops.norm_gated_fwd(d, y, y, w, train=True)
    n = ops.norm_residual_fwd(d, y, None, w, train=True)
    host = torch.empty(1 << 22, dtype=torch.uint8)
    for call in (lambda ws: ops.norm_gated_bwd(d, y, w, f.rstd, y8=f.y8, z8=f.z8, ws=ws),
                 lambda ws: ops.norm_residual_bwd(d, y, w, n.rstd, r8=n.r8, ws=ws),
                 lambda ws: ops.ckpt8_wgrad(y, f.y8, width, ws=ws)):
        assert _status(call, host) == ssm.SSM_ERR_UNSUPPORTED
        call(host.cuda())


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_frozen_scale(io):
    """A scale that is not trained needs no branch in the backward, in ops as in
    the library: without b there is no d_scale, and the rest is the same."""
    rows, width = 33, 200
    b, dh = (R.draw(k, rows, width).to(R.DTYPES[io]).cuda() for k in (1, 2))
    r, dr = (R.draw(k, rows, width).cuda() for k in (3, 4))
    w, scale = (1 + 0.1 * R.draw(5, width)).cuda(), (0.3 + 0.1 * R.draw(6, width)).cuda()
    d = ops.norm_desc(n_rows=rows, width=width, io=io, res_scale=0.7)
    f = ops.norm_residual_fwd(d, b, r, w, scale=scale, train=True)
    args = dict(dr_out=dr, r8=f.r8, scale=scale)
    full = ops.norm_residual_bwd(d, dh, w, f.rstd, b8=f.b8, **args)
    frozen = ops.norm_residual_bwd(d, dh, w, f.rstd, **args)
    assert full.d_scale is not None and frozen.d_scale is None
    want = R.residual_bwd(dh.double().cpu(), dr.double().cpu(), R.kept(f.r_out.cpu()), R.kept(b.cpu()),
                          w.double().cpu(), f.rstd.double().cpu(), scale=scale.double().cpu(), alpha=0.7)
    for name, kind in (("d_r", "f32"), ("d_b", io), ("d_w", "f32")):
        R.check(name, getattr(frozen, name), *want[name], kind, R.COUNT_SUM if name == "d_w" else R.COUNT)
    # asked for by its tensor, it still needs the branch
    assert _status(ops.norm_residual_bwd, d, dh, w, f.rstd, d_scale=torch.empty(width, device="cuda"),
                   **args) == ssm.SSM_ERR_NULL
