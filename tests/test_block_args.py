"""What the operators around the scan make of unusual but possible arguments, on
the CPU: layouts that the library cannot describe are refused by name before
anything is launched."""
import pytest
import torch

import selective_scan_recurrence_amd as ssm
from selective_scan_recurrence_amd import ops


def _status(f, *a, **kw):
    with pytest.raises(ssm.SsmError) as e:
        f(*a, **kw)
    return e.value.status


def _raw_desc(rows, width):
    """A descriptor whose strides are left 0, which stands for dense rows."""
    return ssm.SsmNormDesc(rows, width, 1, 0, 0, 0, 0, ssm.SSM_BF16, ssm.SSM_F32, 1e-5, 1.0, 0, 0)


@pytest.mark.parametrize("width", [1, 40, 96])
def test_expanded_rows_are_refused(width):
    """Rows that share memory (the gradient of a sum over tokens has row stride 0)
    or overlap have no row stride of at least the width."""
    row = torch.zeros(1, width, dtype=torch.bfloat16)
    overlapping = torch.zeros(4 * 96, dtype=torch.bfloat16).as_strided((4, 96), (64, 1))
    ck = torch.zeros(ops.ckpt8_bytes(4, 96), dtype=torch.uint8)
    for bad in (row.expand(4, width), overlapping):
        n = bad.shape[1]
        assert _status(ops.ckpt8_pack, bad) == ssm.SSM_ERR_SHAPE
        assert _status(ops.ckpt8_unpack, ck, 4, n, out=bad) == ssm.SSM_ERR_SHAPE
        assert _status(ops.ckpt8_wgrad, bad, ck, 32) == ssm.SSM_ERR_SHAPE


def test_expanded_rows_do_not_match_a_stride_of_zero():
    d, w = _raw_desc(4, 96), torch.zeros(96)
    dense, row = torch.zeros(4, 96, dtype=torch.bfloat16), torch.zeros(1, 96, dtype=torch.bfloat16)
    bad, bad_f32 = row.expand(4, 96), row.float().expand(4, 96)
    rstd = torch.zeros(4)
    assert _status(ops.norm_gated_fwd, d, bad, dense, w) == ssm.SSM_ERR_SHAPE
    assert _status(ops.norm_gated_bwd, d, bad, w, rstd, y=dense, z=dense) == ssm.SSM_ERR_SHAPE
    assert _status(ops.norm_residual_fwd, d, bad, dense.float(), w) == ssm.SSM_ERR_SHAPE
    assert _status(ops.norm_residual_fwd, d, None, bad_f32, w) == ssm.SSM_ERR_SHAPE
    assert _status(ops.norm_residual_bwd, d, bad, w, rstd, r_out=dense.float()) == ssm.SSM_ERR_SHAPE


def test_a_stride_of_zero_stands_for_dense_rows():
    # a dense tensor on the CPU passes the layout check and is turned away for its device
    d, w = _raw_desc(4, 96), torch.zeros(96)
    dense = torch.zeros(4, 96, dtype=torch.bfloat16)
    assert _status(ops.norm_gated_fwd, d, dense, dense, w) == ssm.SSM_ERR_UNSUPPORTED
    assert _status(ops.norm_residual_fwd, d, dense, dense.float(), w) == ssm.SSM_ERR_UNSUPPORTED
    assert ops._matrix_like(4, 96, 0, torch.float32, "cpu", None).shape == (4, 96)
    # one row has no stride that matters
    assert _status(ops.ckpt8_pack, dense[:1].expand(1, 96)) == ssm.SSM_ERR_UNSUPPORTED


def _on(index, *shape, dtype=torch.float32):
    """A tensor that says it is on GPU index; it has no memory."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        return torch.empty(*shape, dtype=dtype, device=f"cuda:{index}")


IO, RES, U8 = torch.bfloat16, torch.float32, torch.uint8


def _arguments(name):
    """A complete call of ops.<name>: its leading arguments, and its tensors by
    name with their shapes and types."""
    d = ops.norm_desc(n_rows=4, width=96)
    mat, row, col, ck, ws = ((4, 96), IO), ((96,), RES), ((4,), RES), ((ops.ckpt8_bytes(4, 96),), U8), ((1 << 16,), U8)
    stream = ((4, 96), RES)
    return {
        "ckpt8_pack": ([], dict(x=mat, out=ck), {}),
        "ckpt8_unpack": ([], dict(ckpt=ck, out=mat), dict(n_rows=4, width=96)),
        "ckpt8_wgrad": ([], dict(dy=((4, 40), IO), ckpt=ck, dw=((40, 96), RES), ws=ws), dict(width=96)),
        "norm_gated_fwd": ([d], dict(y=mat, z=mat, w=row, out=mat, rstd=col, y8=ck, z8=ck, out8=ck), {}),
        "norm_gated_bwd": ([d], dict(dout=mat, w=row, rstd=col, y=mat, z=mat, d_y=mat, d_z=mat, d_w=row, ws=ws), {}),
        "norm_residual_fwd": ([d], dict(b=mat, r=stream, w=row, w_post=row, scale=row, r_out=stream, h=mat, rstd=col,
                                        rstd_post=col, r8=ck, b8=ck, h8=ck), {}),
        "norm_residual_bwd": ([d], dict(dh=mat, w=row, rstd=col, dr_out=stream, r8=ck, b8=ck, rstd_post=col,
                                        w_post=row, scale=row, d_r=stream, d_b=mat, d_w=row, d_w_post=row,
                                        d_scale=row, ws=ws), {}),
    }[name]


class _Stream:
    """A stream of GPU 1."""
    device_index, cuda_stream = 1, 256


@pytest.mark.parametrize("where", ["cpu", "other", "stream"])
@pytest.mark.parametrize("name", ["ckpt8_pack", "ckpt8_unpack", "ckpt8_wgrad", "norm_gated_fwd", "norm_gated_bwd",
                                  "norm_residual_fwd", "norm_residual_bwd"])
def test_tensors_are_on_the_device_of_the_launch(monkeypatch, name, where):
    """A call launches on its stream's device, without a stream on the current
    one: a tensor in host memory or on another GPU is refused by its name."""
    monkeypatch.setattr(ops, "_current_device", lambda: 0, raising=False)
    lead, tensors, rest = _arguments(name)
    home = 1 if where == "stream" else 0
    for odd in tensors:
        args = {k: _on(home, *shape, dtype=dtype) for k, (shape, dtype) in tensors.items()}
        shape, dtype = tensors[odd]
        args[odd] = torch.empty(*shape, dtype=dtype) if where == "cpu" else _on(1 - home, *shape, dtype=dtype)
        kw = dict(stream=_Stream()) if where == "stream" else {}
        with pytest.raises(ssm.SsmError, match=rf": {odd} is ") as e:
            getattr(ops, name)(*lead, **args, **rest, **kw)
        assert e.value.status == ssm.SSM_ERR_UNSUPPORTED, odd
