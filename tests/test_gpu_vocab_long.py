"""The losses over a vocabulary where it is long for its rows: many parts of d_h's sum,
and several pieces of the vocabulary.  The reference runs on the GPU, in 64 bits."""
import pytest
import torch

import vocab_ref as R
from selective_scan_recurrence_amd import ops
from test_gpu_vocab import compare, run

pytestmark = pytest.mark.gpu


def _on_gpu(*a, **kw):
    return {k: v.cuda() for k, v in R.problem(*a, **kw).items()}


@pytest.mark.parametrize("n,d,v,io,out", [(100, 64, 66000, "bf16", 0.0), (100, 64, 131072, "bf16", 0.5),
                                          (65, 64, 1 << 20, "bf16", 0.0), (128, 128, 131072, "f32", 0.1)])
@pytest.mark.parametrize("both", [True, False])
def test_parts_of_a_long_vocabulary(n, d, v, io, out, both):
    t = _on_gpu(n + v, n, d, v, io, out=out)
    if both:
        return compare(t, io, run(t, io))
    desc = ops.vocab_desc(n_rows=n, width=d, n_vocab=v, io=io)
    f = ops.vocab_ce_fwd(desc, t["h"], t["w"], t["target"])
    g = ops.vocab_ce_bwd(desc, t["h"], t["w"], t["target"], f.loss, f.lse, t["d_loss"], want_w=False)
    want = R.Reference(t["h"], t["w"], io, target=t["target"]).backward(t["d_loss"])
    R.check("d_h", g.d_h, *want["d_h"])
