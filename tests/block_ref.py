"""Plain float64 forms of the operators around the scan (torch on the CPU), with
the magnitudes that their rounding errors scale with.

An f32 evaluation of a sum of terms is off by a small multiple of 2^-24 times
the sum of the terms' magnitudes, however much they cancel.  Each function
returns, next to a result, that magnitude: the formula with every term's
absolute value.  Tests allow COUNT * 2^-24 * magnitude, plus half a step of
the stored type."""
import torch

BLOCK = 32
U = 2.0 ** -24  # half a step of f32
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}

# Roundings that a result may have gathered, in f32 half steps: the argument
# of e^-z is off by |z| log2(e) half steps (12 for the |z| < 8 drawn here), the
# hardware exponential and reciprocal by 2 each; SiLU enters twice (in x and
# as a factor); the mean adds 8 terms in a lane, then log2 of the lanes (10),
# and up to 16 waves: 34; its square root halves that; products and the final
# difference: 10.  2 * 16 + 34 + 17 + 10 < 100.
COUNT = 100
# A column sum adds, beyond its terms' own COUNT, at most 8 rows a lane, 32
# units and 16 + 6 partial rows, for the up to 4096 rows of the tests.
COUNT_SUM = COUNT + 64


def scale_exponent(amax):
    """The smallest k >= -127 with amax <= 448 * 2^k, by stepping k."""
    k = torch.full(amax.shape, -127, dtype=torch.int64)
    for _ in range(260):
        over = amax > 448.0 * torch.pow(torch.tensor(2.0, dtype=torch.float64), k.double())
        if not over.any():
            return k
        k = k + over.long()
    raise AssertionError("no scale")


def e4m3_grid():
    """The 127 non-negative e4m3 values, by their codes 0x00 .. 0x7e."""
    v = []
    for c in range(127):
        e, f = c >> 3, c & 7
        v.append(f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
    return torch.tensor(v, dtype=torch.float64)


def pack_ref(x):
    """(codes [rows][W32] uint8, scale bytes [rows][W32 / 32] uint8) of x
    [rows][width], each code by a search of the e4m3 values: the nearest, the
    even code of two equally near."""
    rows, width = x.shape
    w32 = -(-width // BLOCK) * BLOCK
    v = torch.zeros(rows, w32, dtype=torch.float64)
    v[:, :width] = x.double().cpu()
    v = v.view(rows, -1, BLOCK)
    finite = torch.isfinite(v)
    k = scale_exponent(torch.where(finite, v.abs(), 0.0).amax(-1))
    a = torch.where(finite, v, 0.0).abs() / torch.pow(torch.tensor(2.0, dtype=torch.float64),
                                                      k.double()).unsqueeze(-1)
    grid = e4m3_grid()
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    code = torch.where(up < down, hi, torch.where(up > down, lo, torch.where(hi % 2 == 0, hi, lo)))
    code = torch.where(a == grid[hi], hi, code)
    code = torch.where((k == 120).unsqueeze(-1), code.clamp(max=0x77), code)  # 240: 256 * 2^120 is past f32
    code = torch.where(torch.signbit(v), code + 128, code)
    code = torch.where(finite, code, 127)
    return code.to(torch.uint8).view(rows, w32), (k + 127).to(torch.uint8)


def unpack_ref(codes, scales, width):
    c = codes.long().view(codes.shape[0], -1, BLOCK)
    mag = torch.cat([e4m3_grid(), torch.tensor([float("nan")], dtype=torch.float64)])[c & 127]
    two = torch.pow(torch.tensor(2.0, dtype=torch.float64), scales.double() - 127.0)
    return (torch.where(c >= 128, -mag, mag) * two.unsqueeze(-1)).flatten(1)[:, :width]


def kept(x):
    """x as its 8-bit checkpoint holds it."""
    return unpack_ref(*pack_ref(x), x.shape[1])


def _group(v, g):
    return v.reshape(v.shape[0], g, -1)


def _rstd(u, g, eps):
    return 1.0 / torch.sqrt(_group(u, g).square().mean(-1, keepdim=True) + eps)


def _spread(inv, v, g):
    return (_group(v, g) * inv).reshape(v.shape)


def _mean(v, g):
    return _group(v, g).mean(-1, keepdim=True).expand_as(_group(v, g)).reshape(v.shape)


def silu(z):
    return z * torch.sigmoid(z)


def silu_slope(z):
    s = torch.sigmoid(z)
    return s * (1 + z * (1 - s))


def gated_fwd(y, z, w, g=1, eps=1e-5, after=False):
    gate = torch.ones_like(y) if z is None else silu(z)
    u = y if after else y * gate
    inv = _rstd(u, g, eps)
    return _spread(inv, u, g) * w * (gate if after else 1.0), inv.squeeze(-1)


def gated_bwd(dout, y, z, w, rstd, g=1, after=False):
    """{name: (gradient, magnitude)}; rstd [rows][g] as the forward gave it."""
    inv = rstd.unsqueeze(-1)
    gate = torch.ones_like(y) if z is None else silu(z)
    # SiLU' is a difference of terms of size 1 + |z|
    zz = torch.zeros_like(y) if z is None else z
    s = torch.sigmoid(zz)
    slope, slope_mag = silu_slope(zz), s * (1 + zz.abs())
    x = _spread(inv, y if after else y * gate, g)
    d = dout * gate if after else dout
    dn = d * w
    c, c_mag = _mean(dn * x, g), _mean((dn * x).abs(), g)
    du = _spread(inv, dn - x * c, g)
    du_mag = _spread(inv, dn.abs() + x.abs() * c_mag, g)
    r = {"d_w": ((d * x).sum(0), (d * x).abs().sum(0))}
    if after:
        r["d_y"] = (du, du_mag)
        r["d_z"] = (dout * x * w * slope, (dout * x * w).abs() * slope_mag)
    else:
        r["d_y"] = (du * gate, du_mag * gate.abs())
        r["d_z"] = (du * y * slope, du_mag * y.abs() * slope_mag)
    return r


def residual_fwd(b, r, w, w_post=None, scale=None, alpha=1.0, eps=1e-5):
    """r_out, h, rstd, rstd_post, and the magnitude of r_out."""
    t, inv_post = b, None
    if w_post is not None:
        inv_post = _rstd(b, 1, eps)
        t = _spread(inv_post, b, 1) * w_post
    gain = alpha * (1.0 if scale is None else scale)
    x = r + gain * t
    inv = _rstd(x, 1, eps)
    return (x, _spread(inv, x, 1) * w, inv.reshape(-1),
            None if inv_post is None else inv_post.reshape(-1), r.abs() + (gain * t).abs())


def residual_bwd(dh, dr_out, r_out, b, w, rstd, rstd_post=None, w_post=None, scale=None, alpha=1.0):
    x = r_out * rstd.unsqueeze(-1)
    dn = dh * w
    c, c_mag = _mean(dn * x, 1), _mean((dn * x).abs(), 1)
    d_r = rstd.unsqueeze(-1) * (dn - x * c) + dr_out
    mag = rstd.unsqueeze(-1) * (dn.abs() + x.abs() * c_mag) + dr_out.abs()
    gain = alpha * (torch.ones_like(w) if scale is None else scale)
    dt, dt_mag = gain * d_r, gain.abs() * mag
    r = {"d_r": (d_r, mag), "d_w": ((dh * x).sum(0), (dh * x).abs().sum(0))}
    if w_post is None:
        r["d_b"] = (dt, dt_mag)
        t = b
    else:
        inv = rstd_post.unsqueeze(-1)
        v = b * inv
        t = v * w_post
        dm, dm_mag = dt * w_post, dt_mag * w_post.abs()
        r["d_b"] = (inv * (dm - v * _mean(dm * v, 1)),
                    inv * (dm_mag + v.abs() * _mean(dm_mag * v.abs(), 1)))
        r["d_w_post"] = ((dt * v).sum(0), (dt_mag * v.abs()).sum(0))
    if scale is not None:
        r["d_scale"] = ((alpha * d_r * t).sum(0), (abs(alpha) * mag * t.abs()).sum(0))
    return r


def check(what, got, want, mag, io, count=COUNT):
    """got (device tensor in io) against want, within half a step of io and
    count f32 half steps of the magnitude."""
    got = got.detach().double().cpu().reshape(want.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    slack = (got - want).abs() - (HALF_STEP[io] * want.abs() + count * U * mag)
    if not (slack <= 0).all():
        at = int(slack.argmax())
        raise AssertionError(f"{what}: {int((slack > 0).sum())} of {slack.numel()} outside; worst at {at}: "
                             f"got {got.flatten()[at]!r}, want {want.flatten()[at]!r}")


def draw(seed, *shape, std=1.0, limit=7.5):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * std).clamp(-limit, limit)


def strided(x, pad, dtype, device="cuda"):
    """x on the device as the first columns of rows pad elements longer (the
    rest a recognisable filler)."""
    rows, width = x.shape
    t = torch.full((rows, width + pad), 77.0, dtype=dtype, device=device)
    t[:, :width] = x.to(dtype).to(device)
    return t[:, :width]


def padding_untouched(t):
    """Whether the filler past t's columns is still there."""
    base = t._base if t._base is not None else t
    return bool((base[:, t.shape[1]:] == 77.0).all())
