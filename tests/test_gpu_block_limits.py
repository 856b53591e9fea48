"""The operators around the scan at the far ends of what they take."""
import pytest
import torch

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
