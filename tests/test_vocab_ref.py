"""The 64-bit reference of the losses over a vocabulary, on the CPU: its gradients
are those of central differences, its losses those of closed forms."""
import math

import pytest
import torch

import vocab_ref as R


def _loss(t, kw, h, w):
    r = R.Reference(h, w, "f32", **{k: v for k, v in t.items() if k in ("target", "top_id", "top_logit")}, **kw)
    return r


@pytest.mark.parametrize("top,as_it_stands", [(0, False), (5, False), (5, True)])
def test_gradients_against_differences(top, as_it_stands):
    t = R.problem(top, 6, 7, 11, "f32", top=top, out=0.3)
    h, w = t["h"].double(), t["w"].double()
    kw = dict(scale=0.8, top_scale=0.6)
    if as_it_stands:
        kw["top_lse"] = torch.logsumexp(t["top_logit"] * 0.6, 1) + 0.3
    d_lse = torch.randn(6, generator=torch.Generator().manual_seed(3), dtype=torch.float64)

    def total(h, w):
        r = _loss(t, kw, h, w).forward()
        return float((r["loss"][0] * t["d_loss"].double() + r["lse"][0] * d_lse).sum())

    grads = _loss(t, kw, h, w).backward(t["d_loss"], d_lse)
    eps = 1e-6
    for name, x in (("d_h", h), ("d_w", w)):
        got = grads[name][0]
        for at in range(x.numel()):
            i, j = divmod(at, x.shape[1])
            up, down = x.clone(), x.clone()
            up[i, j] += eps
            down[i, j] -= eps
            num = (total(up, w) - total(down, w) if name == "d_h" else total(h, up) - total(h, down)) / (2 * eps)
            assert abs(num - float(got[i, j])) < 1e-7, (name, i, j)


def test_zero_weights_spread_evenly():
    t = R.problem(1, 5, 8, 64, "f32")
    r = R.Reference(t["h"], torch.zeros(64, 8), "f32", target=t["target"]).forward()
    assert torch.allclose(r["loss"][0], torch.full((5,), math.log(64), dtype=torch.float64))


def test_one_entry_is_cross_entropy():
    t = R.problem(2, 9, 8, 30, "f32", out=0.4)
    ce = R.Reference(t["h"], t["w"], "f32", target=t["target"])
    kd = R.Reference(t["h"], t["w"], "f32", top_id=t["target"][:, None], top_logit=torch.randn(9, 1))
    assert torch.equal(ce.loss * ce.keep, kd.loss * kd.keep)
    a, b = ce.backward(t["d_loss"]), kd.backward(t["d_loss"])
    assert all(torch.allclose(a[k][0], b[k][0], atol=1e-15) for k in a)
