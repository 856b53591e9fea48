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
