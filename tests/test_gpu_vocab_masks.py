"""Distillation from teacher's logits that hold the lowest finite value, as masked
logits do, or the highest with a negative scale: such an entry has no mass beside
others, and entries that all hold it share the mass."""
import pytest
import torch

import vocab_ref as R
from test_gpu_vocab import run

pytestmark = pytest.mark.gpu

LOWEST = {"f32": torch.finfo(torch.float32).min, "bf16": torch.finfo(torch.bfloat16).min}


class Reference(R.Reference):
    """With a bound on p that holds for any finite logits.  The argument of p's exponential
    is a difference, formed by a rounding of the difference and two of its products with
    constants: it is off by 3 of its own half steps, for which 4 steps of the largest
    difference stand, whatever the logits' own size.  An entry whose p is 0 has no part
    in the loss; p below TINY may count as 0, which is far below a step of the rest."""

    def __init__(self, h, w, io, *, top_id, top_logit, top_lse=None, scale=1.0, top_scale=1.0):
        super().__init__(h, w, io, top_id=top_id, top_logit=top_logit, top_lse=top_lse, scale=scale,
                         top_scale=top_scale)
        t = top_logit.double() * top_scale
        base = torch.where(self.there, t, -float("inf")).amax(1) if top_lse is None else top_lse.double()
        far = (t - base[:, None])[self.there & (self.p > 0)].abs()
        self.p_err = R.STEP * (4 * (float(far.max()) if len(far) else 0.0) + top_id.shape[1] + 16)
        each = torch.where(self.p > 0, torch.log(torch.where(self.p > 0, self.p, 1.0)), 0.0) - self.logq
        self.loss_err = (self.p * (self.logq_err + self.p_err + R.STEP * 8 * (1 + each.abs()))).sum(1) + \
            (self.p * each.abs()).sum(1) * self.p_err


def compare(t, io, **kw):
    got = run(t, io, **kw)
    ref = Reference(t["h"], t["w"], io, top_id=t["top_id"], top_logit=t["top_logit"], **kw)
    assert bool(torch.isfinite(ref.loss).all())
    for name, (value, err) in {**ref.forward(), **ref.backward(t["d_loss"])}.items():
        R.check(name, got[name], value, err)


def _masked(n, top, io, where, value):
    """Some entries of a row, or all entries of every third row, hold `value`."""
    t = R.problem(n + top, n, 64, 300, io, top=top, out=0.2)
    if where == "some":
        t["top_logit"][:, 1::3] = value
    else:
        t["top_logit"][::3] = value
    return t


def _lse(t, top_scale):
    there = t["top_id"] >= 0
    s = torch.where(there, t["top_logit"].double() * top_scale, -float("inf"))
    return torch.where(there.any(1), torch.logsumexp(s, 1), 0.0).float()


@pytest.mark.parametrize("stands", [False, True])
@pytest.mark.parametrize("where", ["some", "all"])
@pytest.mark.parametrize("lowest", ["f32", "bf16"])
@pytest.mark.parametrize("n,io", [(9, "bf16"), (40, "f32"), (140, "bf16"), (140, "f32"), (600, "bf16"), (4200, "bf16")])
def test_lowest_logits(n, io, lowest, where, stands):
    t = _masked(n, 5, io, where, LOWEST[lowest])
    compare(t, io, **(dict(top_lse=_lse(t, 1.0)) if stands else {}))


@pytest.mark.parametrize("top_scale", [-1.0, -0.25, 0.0, 1e-38, 0.5, 2.0, 1e30])
@pytest.mark.parametrize("where", ["some", "all"])
@pytest.mark.parametrize("n", [9, 140])
def test_scales_of_extreme_logits(n, where, top_scale):
    value = LOWEST["f32"] if top_scale >= 0 else -LOWEST["f32"]
    t = _masked(n, 4, "f32", where, value)
    if top_scale == 1e30:  # the rest a step of 1e30 apart: one entry has all of the mass
        t["top_logit"] = torch.where(t["top_logit"] == value, value, torch.round(t["top_logit"]))
    compare(t, "f32", top_scale=top_scale)


@pytest.mark.parametrize("n", [9, 140])
def test_lowest_and_highest(n):
    """Both ends in a row: their difference passes the largest f32 value."""
    t = _masked(n, 6, "bf16", "some", LOWEST["f32"])
    t["top_logit"][:, 2] = -LOWEST["f32"]
    compare(t, "bf16")


@pytest.mark.parametrize("n", [9, 140])
def test_one_lowest_entry(n):
    """A row's only entry has all of the mass, whatever it holds."""
    t = R.problem(n, n, 64, 300, "f32", top=1)
    t["top_logit"][:] = LOWEST["f32"]
    compare(t, "f32")


@pytest.mark.parametrize("n", [9, 140])
def test_same_id_with_and_without_mass(n):
    t = R.problem(n, n, 64, 300, "f32", top=6)
    t["top_id"][:, 3] = t["top_id"][:, 1] = t["top_id"][:, 0]
    t["top_logit"][:, 1] = LOWEST["f32"]
    compare(t, "f32")
