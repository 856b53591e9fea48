"""Calls of the losses over a vocabulary that their description allows: tensors that
start inside others, outputs that are not wanted, a workspace that holds anything, a
vocabulary of one or two."""
import pytest
import torch

import selective_scan_recurrence_amd as ssm
import vocab_ref as R
from selective_scan_recurrence_amd import ops
from test_gpu_vocab import compare, run

pytestmark = pytest.mark.gpu


def _inside(x, dtype, start):
    """x on the GPU in a buffer, `start` elements in, rows 64 elements apart or a multiple."""
    rows, width = x.shape
    ld = (width + 63) // 64 * 64
    buf = torch.full((rows * ld + 64,), 77.0, dtype=dtype, device="cuda")
    view = buf[start:start + rows * ld].view(rows, ld)[:, :width]
    view.copy_(x.to(dtype))
    return view, buf


@pytest.mark.parametrize("start", [1, 2, 4])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,d,top", [(5, 64, 0), (40, 128, 3), (140, 64, 3), (300, 128, 0), (70, 100, 0)])
def test_tensors_inside_others(n, d, top, io, start):
    """Their rows' strides would allow wide loads, their addresses do not."""
    v, dt = 300, R.DTYPES[io]
    t = R.problem(n + start, n, d, v, io, top=top, out=0.2)
    ld = (d + 63) // 64 * 64
    desc = ops.vocab_desc(n_rows=n, width=d, n_vocab=v, n_top=top, io=io, dw=io, ld_h=ld, ld_w=ld)
    (h, _), (w, _) = _inside(t["h"], dt, start), _inside(t["w"], dt, start)
    (d_h, all_h), (d_w, all_w) = _inside(torch.zeros(n, d), dt, start), _inside(torch.zeros(v, d), dt, start)
    g = {k: x.cuda() for k, x in t.items()}
    if top:
        f = ops.vocab_kd_fwd(desc, h, w, g["top_id"], g["top_logit"])
        ops.vocab_kd_bwd(desc, h, w, g["top_id"], g["top_logit"], f.logq, f.lse, g["d_loss"], d_h=d_h, d_w=d_w)
    else:
        f = ops.vocab_ce_fwd(desc, h, w, g["target"])
        ops.vocab_ce_bwd(desc, h, w, g["target"], f.loss, f.lse, g["d_loss"], d_h=d_h, d_w=d_w)
    compare(t, io, {"loss": f.loss, "lse": f.lse, "logq": f.logq, "d_h": d_h, "d_w": d_w}, dw=io)
    for buf, rows in ((all_h, n), (all_w, v)):
        kept = torch.ones_like(buf, dtype=torch.bool)
        kept[start:start + rows * ld].view(rows, ld)[:, :d] = False
        assert bool((buf[kept] == 77.0).all())


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n", [5, 140, 600])
def test_outputs_that_are_not_wanted(n, io):
    for top, wanted in ((0, ["loss", "lse"]), (3, ["loss", "lse", "logq"])):
        t = {k: x.cuda() for k, x in R.problem(n + top, n, 64, 300, io, top=top, out=0.2).items()}
        desc = ops.vocab_desc(n_rows=n, width=64, n_vocab=300, n_top=top, io=io)
        ws = ops.vocab_workspace(desc, False)

        def call(names):
            out = {k: torch.full((n, top) if k == "logq" else (n,), 7.0, device="cuda") if k in names else None
                   for k in wanted}
            if top:
                ssm.ssm_vocab_kd_fwd(desc, t["h"], t["w"], t["top_id"], t["top_logit"], None, out["loss"], out["lse"],
                                     out["logq"], None, ws, ws.numel(), torch.cuda.current_stream())
            else:
                ssm.ssm_vocab_ce_fwd(desc, t["h"], t["w"], t["target"], out["loss"], out["lse"], None, ws, ws.numel(),
                                     torch.cuda.current_stream())
            return out

        everything = call(wanted)
        for some in [[k] for k in wanted] + [[]]:
            for name, x in call(some).items():
                assert x is None or torch.equal(x, everything[name]), (top, some, name)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,d,v,top", [(5, 72, 700, 0), (40, 64, 300, 3), (140, 72, 700, 3), (600, 200, 2100, 0),
                                       (3000, 70, 256, 0), (70, 65, 9000, 2)])
def test_a_workspace_holds_anything(n, d, v, top, io):
    """The results of a workspace of NaN (and of numbers past every count) are those of
    one of zeros."""
    t = R.problem(n + v, n, d, v, io, top=top, out=0.3)
    desc = ops.vocab_desc(n_rows=n, width=d, n_vocab=v, n_top=top, io=io)
    got = []
    for fill in (0x00, 0xFF, 0x7F):
        ws = torch.full_like(ops.vocab_workspace(desc, True), fill)
        got.append(run(t, io, ws=ws))
    for other in got[1:]:
        for name, x in got[0].items():
            assert x is None or torch.equal(x, other[name]), name


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n", [3, 64, 65, 300])
@pytest.mark.parametrize("v", [1, 2])
@pytest.mark.parametrize("top", [0, 4])
def test_a_vocabulary_of_one_or_two(n, v, top, io):
    t = R.problem(n + v, n, 40, v, io, top=top, out=0.2)
    compare(t, io, run(t, io))
