"""Refusals and sizes of the operators around the scan, on the CPU: every bad
argument is turned away on the host with its documented status before a
launch.  Pointers are small integers that are never followed."""
import pytest
import torch

import selective_scan_recurrence_amd as ssm
from selective_scan_recurrence_amd import ops

BIG = 1 << 40


def _status(f, *a, **kw):
    with pytest.raises(ssm.SsmError) as e:
        f(*a, **kw)
    return e.value.status


def _desc(**kw):
    return ops.norm_desc(**{**dict(n_rows=4, width=96), **kw})


def _gated_fwd(d, **kw):
    a = dict(y=256, z=256, w=256, out=256, rstd=256, y8=None, z8=None, out8=None)
    a.update(kw)
    return ssm.ssm_norm_gated_fwd(d, *a.values(), stream=0)


def _gated_bwd(d, **kw):
    a = dict(dout=256, y=256, z=256, y8=None, z8=None, w=256, rstd=256, d_y=256, d_z=256, d_w=256,
             workspace=256, workspace_bytes=BIG)
    a.update(kw)
    return ssm.ssm_norm_gated_bwd(d, *a.values(), stream=0)


def _residual_fwd(d, **kw):
    a = dict(b=256, r=256, w_post=None, scale=None, w=256, r_out=256, h=256, rstd=256, rstd_post=None,
             r8=None, b8=None, h8=None)
    a.update(kw)
    return ssm.ssm_norm_residual_fwd(d, *a.values(), stream=0)


def _residual_bwd(d, **kw):
    a = dict(dh=256, dr_out=256, r_out=256, r8=None, b=None, b8=None, w_post=None, scale=None, w=256,
             rstd=256, rstd_post=None, d_r=256, d_b=256, d_w=256, d_w_post=None, d_scale=None,
             workspace=256, workspace_bytes=BIG)
    a.update(kw)
    return ssm.ssm_norm_residual_bwd(d, *a.values(), stream=0)


NORMS = [_gated_fwd, _gated_bwd, _residual_fwd, _residual_bwd]


@pytest.mark.parametrize("call", NORMS)
@pytest.mark.parametrize("field,value", [
    ("n_rows", -1), ("n_rows", 1 << 31), ("width", 0), ("width", -8), ("width", 1 << 31), ("width", (1 << 22) + 1),
    ("width", 40000), ("n_group", 0), ("n_group", 5), ("n_group", 192), ("ld_x", 95), ("ld_z", 1),
    ("ld_res", -96), ("ld_out", 95), ("ld_x", 1 << 61), ("eps", 0.0), ("eps", -1e-5),
    ("eps", float("nan")), ("eps", float("inf")), ("res_scale", float("inf")),
    ("res_scale", float("nan")), ("flags", 2), ("reserved", 1),
])
def test_bad_descriptor(call, field, value):
    d = _desc()
    setattr(d, field, value)
    assert _status(call, d) == ssm.SSM_ERR_SHAPE
    assert ssm.ssm_norm_bwd_workspace_bytes(d) == 0


@pytest.mark.parametrize("call", NORMS)
@pytest.mark.parametrize("field", ["io_dtype", "res_dtype"])
def test_bad_dtype(call, field):
    d = _desc()
    setattr(d, field, 5)
    assert _status(call, d) == ssm.SSM_ERR_DTYPE


def test_row_group_product_is_bounded():
    assert _status(_gated_fwd, _desc(n_rows=1 << 28, n_group=96)) == ssm.SSM_ERR_SHAPE


def test_residual_takes_one_group_and_no_gate():
    for call in (_residual_fwd, _residual_bwd):
        assert _status(call, _desc(n_group=2)) == ssm.SSM_ERR_SHAPE
        assert _status(call, _desc(gate_after=True)) == ssm.SSM_ERR_SHAPE
        assert _status(call, _desc(io="f32", res="bf16")) == ssm.SSM_ERR_UNSUPPORTED


@pytest.mark.parametrize("call,names", [
    (_gated_fwd, ["y", "w", "out"]),
    (_gated_bwd, ["dout", "y", "w", "rstd", "workspace"]),
    (_residual_fwd, ["w", "h"]),
    (_residual_bwd, ["dh", "r_out", "w", "rstd", "workspace"]),
])
def test_missing_pointer(call, names):
    for name in names:
        assert _status(call, _desc(), **{name: None}) == ssm.SSM_ERR_NULL, name


def test_missing_partner():
    null = ssm.SSM_ERR_NULL
    assert _status(_gated_fwd, _desc(), z=None, z8=256) == null
    assert _status(_gated_bwd, _desc(), z=None) == null              # d_z without z
    assert _status(_residual_fwd, _desc(), b=None, r=None) == null
    for name in ("w_post", "scale", "b8"):
        assert _status(_residual_fwd, _desc(), b=None, **{name: 256}) == null
    assert _status(_residual_fwd, _desc(), rstd_post=256) == null    # without w_post
    assert _status(_residual_bwd, _desc(), w_post=256, rstd_post=256) == null  # without b
    assert _status(_residual_bwd, _desc(), d_scale=256) == null
    assert _status(_residual_bwd, _desc(), w_post=256, b=256) == null          # without rstd_post
    assert _status(_residual_bwd, _desc(), d_w_post=256) == null               # without w_post


def test_tensor_and_checkpoint_together():
    both = ssm.SSM_ERR_UNSUPPORTED
    assert _status(_gated_bwd, _desc(), y8=256) == both
    assert _status(_gated_bwd, _desc(), z8=256) == both
    assert _status(_residual_bwd, _desc(), r8=256) == both
    assert _status(_residual_bwd, _desc(), b=256, b8=256) == both


def test_checkpoint_blocks_stay_in_a_group():
    d = _desc(n_group=2)  # 48 columns a group
    for name in ("y8", "z8", "out8"):
        assert _status(_gated_fwd, d, **{name: 256}) == ssm.SSM_ERR_UNSUPPORTED
    assert _status(_gated_bwd, d, y=None, y8=256) == ssm.SSM_ERR_UNSUPPORTED


@pytest.mark.parametrize("call,names", [
    (_gated_fwd, ["w", "rstd"]), (_gated_bwd, ["w", "rstd", "d_w", "workspace"]),
    (_residual_fwd, ["w", "rstd", "r", "r_out"]),
    (_residual_bwd, ["w", "rstd", "r_out", "d_r", "dr_out", "workspace"]),
])
def test_misaligned(call, names):
    for name in names:
        assert _status(call, _desc(), **{name: 258}) == ssm.SSM_ERR_ALIGN, name
    assert _status(call, _desc(), w=258) == ssm.SSM_ERR_ALIGN


def test_misaligned_checkpoint():
    assert _status(_gated_fwd, _desc(), y8=264) == ssm.SSM_ERR_ALIGN
    assert _status(_residual_fwd, _desc(), h8=264) == ssm.SSM_ERR_ALIGN
    assert _status(_residual_bwd, _desc(), r_out=None, r8=264) == ssm.SSM_ERR_ALIGN


def test_short_workspace():
    for call in (_gated_bwd, _residual_bwd):
        need = ssm.ssm_norm_bwd_workspace_bytes(_desc(n_rows=100))
        assert need > 0
        assert _status(call, _desc(n_rows=100), workspace_bytes=need - 1) == ssm.SSM_ERR_WORKSPACE


def test_no_rows_need_no_matrices():
    # nothing is launched for the forwards; the checks pass with NULL matrices
    d = _desc(n_rows=0)
    _gated_fwd(d, y=None, z=None, out=None, rstd=None)
    _residual_fwd(d, b=None, r=None, r_out=None, h=None, rstd=None)
    ssm.ssm_ckpt8_pack(None, 0, 0, 96, 1, None, stream=0)
    ssm.ssm_ckpt8_unpack(None, None, 0, 0, 96, 1, stream=0)


@pytest.mark.parametrize("width,w32", [(1, 32), (31, 32), (32, 32), (33, 64), (515, 544), (5120, 5120)])
def test_checkpoint_bytes(width, w32):
    assert ssm.ssm_ckpt8_bytes(7, width) == (7 * w32 + 7 * w32 // 32, 7 * w32)
    assert ssm.ssm_ckpt8_bytes(0, width) == (0, 0)


def test_checkpoint_refusals():
    def pack(x=256, ld=96, rows=4, width=96, dtype=1, ckpt=256):
        return ssm.ssm_ckpt8_pack(x, ld, rows, width, dtype, ckpt, stream=0)

    def unpack(x=256, ld=96, rows=4, width=96, dtype=1, ckpt=256):
        return ssm.ssm_ckpt8_unpack(ckpt, x, ld, rows, width, dtype, stream=0)

    for f in (pack, unpack):
        assert _status(f, dtype=2) == ssm.SSM_ERR_DTYPE
        for kw in (dict(rows=-1), dict(width=0), dict(width=1 << 31), dict(ld=95), dict(ld=-1),
                   dict(rows=1 << 50), dict(ld=1 << 62)):
            assert _status(f, **kw) == ssm.SSM_ERR_SHAPE, kw
        assert _status(f, x=None) == ssm.SSM_ERR_NULL
        assert _status(f, ckpt=None) == ssm.SSM_ERR_NULL
        assert _status(f, x=257) == ssm.SSM_ERR_ALIGN
        assert _status(f, x=258, dtype=0) == ssm.SSM_ERR_ALIGN
        assert _status(f, ckpt=264) == ssm.SSM_ERR_ALIGN
    for rows, width in ((-1, 96), (4, 0), (4, 1 << 31), (1 << 50, 96)):
        assert ssm.ssm_ckpt8_bytes(rows, width) == (0, 0)


def test_wgrad_refusals():
    def wgrad(dy=256, ld=40, ckpt=256, dw=256, rows=64, width=96, n_out=40, dtype=1, acc=0, ws=256,
              ws_bytes=BIG):
        return ssm.ssm_ckpt8_wgrad(dy, ld, ckpt, dw, rows, width, n_out, dtype, acc, ws, ws_bytes,
                                   stream=0)

    assert _status(wgrad, dtype=9) == ssm.SSM_ERR_DTYPE
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(width=0), dict(n_out=0), dict(ld=39),
               dict(width=(1 << 22) + 1), dict(n_out=(1 << 22) + 1), dict(ld=1 << 60)):
        assert _status(wgrad, **kw) == ssm.SSM_ERR_SHAPE, kw
    for name in ("dy", "ckpt", "dw"):
        assert _status(wgrad, **{name: None}) == ssm.SSM_ERR_NULL
    for kw in (dict(dy=257), dict(ckpt=264), dict(dw=258), dict(dy=258, dtype=0)):
        assert _status(wgrad, **kw) == ssm.SSM_ERR_ALIGN, kw
    need = ssm.ssm_ckpt8_wgrad_workspace_bytes(8192, 512, 512, 1)
    if need:
        assert _status(wgrad, rows=8192, width=512, n_out=512, ld=512, ws_bytes=need - 1) == \
            ssm.SSM_ERR_WORKSPACE
        assert _status(wgrad, rows=8192, width=512, n_out=512, ld=512, ws=None) == ssm.SSM_ERR_NULL


@pytest.mark.parametrize("dtype", [0, 1])
def test_wgrad_workspace(dtype):
    """Whole partials of dw, none where one workgroup a tile takes all rows."""
    for rows in (0, 1, 63, 64, 65, 777, 8192, 100000, (1 << 31) - 2000):
        for width, n_out in ((1, 1), (515, 130), (2560, 10576), (1 << 22, 3)):
            n = ssm.ssm_ckpt8_wgrad_workspace_bytes(rows, width, n_out, dtype)
            counts = [0, *range(2, min(512, -(-rows // 64)) + 1)]  # rounded up to 256 bytes
            assert n in {-(-4 * width * n_out * k // 256) * 256 for k in counts}, (rows, width, n_out)


def test_tensors_are_checked():
    """ops: a tensor of another shape, stride, type or device than the
    descriptor says is refused by its name."""
    d = ops.norm_desc(n_rows=4, width=96)
    y = torch.zeros(4, 96, dtype=torch.bfloat16)
    w = torch.zeros(96)
    assert _status(ops.norm_gated_fwd, d, y, y, w) == ssm.SSM_ERR_UNSUPPORTED  # on the CPU
    assert _status(ops.norm_gated_fwd, d, y.float(), y, w) == ssm.SSM_ERR_DTYPE
    assert _status(ops.norm_residual_fwd, d, y, y.float(), w) == ssm.SSM_ERR_UNSUPPORTED
    assert _status(ops._matrix, "here", "r", y, 4, 96, 96, torch.float32) == ssm.SSM_ERR_DTYPE
    wide = torch.zeros(4, 128, dtype=torch.bfloat16)
    for bad in (y[:3], y[:, :95], wide[:, :96], y.t().contiguous().t(), y.view(2, 2, 96)):
        assert _status(ops.norm_gated_fwd, d, bad, y, w) == ssm.SSM_ERR_SHAPE
    for bad in (w[:95], torch.zeros(192)[::2]):
        assert _status(ops.norm_gated_bwd, ops.norm_desc(n_rows=0, width=96), y[:0], bad, w) in \
            (ssm.SSM_ERR_SHAPE, ssm.SSM_ERR_UNSUPPORTED)
        assert _status(ops._dense, "here", "w", bad, 96, torch.float32) == ssm.SSM_ERR_SHAPE
    assert _status(ops.ckpt8_pack, y.t().contiguous().t()) == ssm.SSM_ERR_SHAPE
    short = torch.zeros(ops.ckpt8_bytes(4, 96) - 1, dtype=torch.uint8)
    assert _status(ops.ckpt8_unpack, short, 4, 96) == ssm.SSM_ERR_SHAPE
    assert _status(ops.ckpt8_pack, y) == ssm.SSM_ERR_UNSUPPORTED
    assert _status(ops.ckpt8_pack, y.half()) == ssm.SSM_ERR_DTYPE
    assert _status(ops.ckpt8_wgrad, y, torch.zeros(1, dtype=torch.uint8), 32) == ssm.SSM_ERR_UNSUPPORTED
