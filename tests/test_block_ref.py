"""The float64 forms of tests/block_ref.py pinned on the CPU: gradients by
central differences of the forward, the 8-bit format by torch's own e4m3 cast
and by closed forms."""
import math

import pytest
import torch

import block_ref as R


def _differences(f, x, d, eps=1e-6):
    """d/dt f(x + t d) at 0, by central differences."""
    return (f(x + eps * d) - f(x - eps * d)) / (2 * eps)


def _dot(a, b):
    return float((a * b).sum())


def _near(a, b):
    assert math.isclose(a, b, rel_tol=1e-6, abs_tol=1e-8), (a, b)


@pytest.mark.parametrize("groups", [1, 3])
@pytest.mark.parametrize("after", [False, True])
@pytest.mark.parametrize("gated", [True, False])
def test_gated_gradient_by_differences(groups, after, gated):
    y, z, w = (R.draw(k, 4, 12).double() for k in (1, 2, 3))
    z, w = z if gated else None, 1 + 0.2 * w[0]
    d, way = R.draw(4, 4, 12).double(), R.draw(5, 4, 12).double()
    rstd = R.gated_fwd(y, z, w, groups, 1e-3, after)[1]
    grads = R.gated_bwd(d, y, z, w, rstd, groups, after)

    def out(y, z, w):
        return (R.gated_fwd(y, z, w, groups, 1e-3, after)[0] * d).sum()

    _near(_dot(grads["d_y"][0], way), float(_differences(lambda v: out(v, z, w), y, way)))
    if gated:
        _near(_dot(grads["d_z"][0], way), float(_differences(lambda v: out(y, v, w), z, way)))
    _near(_dot(grads["d_w"][0], way[0]), float(_differences(lambda v: out(y, z, v), w, way[0])))
    for g, mag in grads.values():
        assert (g.abs() <= mag * (1 + 1e-12)).all()


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("scaled", [False, True])
def test_residual_gradient_by_differences(post, scaled):
    b, r, dh, dr, way = (R.draw(k, 5, 9).double() for k in range(11, 16))
    w, wp, sc = (1 + 0.3 * R.draw(k, 9).double() for k in (16, 17, 18))
    wp, sc = wp if post else None, sc if scaled else None
    _, _, rstd, rstd_post, _ = R.residual_fwd(b, r, w, wp, sc, 0.7, 1e-3)

    def loss(b, r, w, wp, sc):
        x, h, _, _, _ = R.residual_fwd(b, r, w, wp, sc, 0.7, 1e-3)
        return (x * dr).sum() + (h * dh).sum()

    x = R.residual_fwd(b, r, w, wp, sc, 0.7, 1e-3)[0]
    g = R.residual_bwd(dh, dr, x, b, w, rstd, rstd_post, wp, sc, 0.7)
    _near(_dot(g["d_r"][0], way), float(_differences(lambda v: loss(b, v, w, wp, sc), r, way)))
    _near(_dot(g["d_b"][0], way), float(_differences(lambda v: loss(v, r, w, wp, sc), b, way)))
    _near(_dot(g["d_w"][0], way[0]), float(_differences(lambda v: loss(b, r, v, wp, sc), w, way[0])))
    if post:
        _near(_dot(g["d_w_post"][0], way[0]), float(_differences(lambda v: loss(b, r, w, v, sc), wp, way[0])))
    if scaled:
        _near(_dot(g["d_scale"][0], way[0]), float(_differences(lambda v: loss(b, r, w, wp, v), sc, way[0])))
    for v, mag in g.values():
        assert (v.abs() <= mag * (1 + 1e-12)).all()


def test_codes_are_torchs_e4m3():
    assert torch.equal(R.e4m3_grid().float(),
                       torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float())
    x = R.draw(21, 64, 96, limit=100.0)
    x[0] = x[0].bfloat16().float()  # ties
    codes, scales = R.pack_ref(x)
    two = torch.pow(2.0, scales.double() - 127).repeat_interleave(32, 1)
    want = (x.double() / two).float().to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(codes, want)


def test_scale_borders():
    # 448 * 2^k is the last amax of k; one step above needs k + 1
    for k in (-127, -40, 0, 7, 119):
        top = torch.tensor([448.0 * 2.0 ** k], dtype=torch.float64)
        assert int(R.scale_exponent(top)) == k
        assert int(R.scale_exponent(top * (1 + 2.0 ** -20))) == k + 1
    assert int(R.scale_exponent(torch.zeros(1, dtype=torch.float64))) == -127
    x = torch.tensor([[448.0, -448.0, 1.0, 0.0, -0.0, 2.0 ** -10, 2.0 ** -9, 3 * 2.0 ** -10]])
    codes, scales = R.pack_ref(x)
    assert int(scales) == 127
    # 2^-10 is half a step: the even code 0; 3 * 2^-10 lies between codes 1 and 2
    assert codes[0, :8].tolist() == [126, 254, 0x38, 0, 128, 0, 1, 2]
    assert not codes[0, 8:].any()


def test_kept_is_within_half_a_step():
    x = R.draw(22, 50, 70, limit=50.0) * torch.logspace(-3, 3, 70)
    got = R.kept(x)
    _, scales = R.pack_ref(x)
    low = torch.pow(2.0, scales.double() - 127 - 10).repeat_interleave(32, 1)[:, :70]
    assert ((got - x.double()).abs() <= torch.maximum(x.double().abs() * 2.0 ** -4, low)).all()


def test_values_that_are_not_finite():
    x = R.draw(23, 2, 64)
    x[0, 3], x[0, 5], x[1, 40] = float("nan"), float("inf"), -float("inf")
    got = R.kept(x)
    bad = ~torch.isfinite(x)
    assert torch.isnan(got[bad]).all()
    assert torch.equal(got[~bad], R.kept(torch.where(bad, 0.0, x))[~bad])
