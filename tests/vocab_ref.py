"""Plain 64-bit implementation of the losses over a vocabulary and of their
gradients, and how far the kernels may be from it.

Tolerances, before any run: STEP = 2^-23 is a whole step of f32, since the
matrix unit may cut off where it does not round.  A sum of n products is off by
at most a step of its magnitude for each of the additions that it makes one
after the other: one for every 8 products (the fewest that the matrix unit takes
at once), six runs over them in f32, and a few to join parts (a sum's p parts have
128 products or more each: a part's additions and p joins, n/8p + p with p <= n/128
are no more than n/8 for p >= 2); in f32 its products are also off by 2^-21 each.  From the logits' error follow those of the
statistics, of g (an exponential is off by as much, relative to itself, as its
argument is), and of the products with g, which is rounded to its type first.
Below TINY = 2^-126 f32 values may count as zero: an exponential and then g, so
that g is off by (|coef| + 1) TINY more, and each of a sum's n products, n TINY.
"""
import torch

STEP = 2.0 ** -23
TINY = 2.0 ** -126
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
# half a step of the type relative to the value
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def _chain(n, io):
    """Relative error of a sum of n products, of its magnitude."""
    return STEP * ((n / 8 + 12) * (6 if io == "f32" else 1)) + (2.0 ** -21 if io == "f32" else 0.0)


def teacher(top_id, top_logit, top_scale, top_lse):
    """p [n][k] in 64 bits and which entries are there."""
    there = (top_id >= 0) & (top_logit != -float("inf"))
    t = torch.where(there, top_logit.double() * top_scale, -float("inf"))
    if top_lse is None:
        high = t.amax(1, keepdim=True)
        p = torch.exp(t - torch.where(there.any(1, keepdim=True), high, 0.0))
        p = p / torch.where(there.any(1, keepdim=True), p.sum(1, keepdim=True), 1.0)
    else:
        p = torch.exp(t - top_lse.double()[:, None])
    return torch.where(there, p, 0.0), there


class Reference:
    """h [n][d] and w [v][d] as the kernel has them (any float type, on the CPU)."""

    def __init__(self, h, w, io, *, target=None, top_id=None, top_logit=None, top_lse=None, scale=1.0,
                 top_scale=1.0):
        h, w = h.double(), w.double()
        n, v = h.shape[0], w.shape[0]
        if target is not None:
            ids, there = target.long()[:, None], (target >= 0)[:, None]
            p, p_err = there.double(), 0.0
        else:
            p, there = teacher(top_id, top_logit, top_scale, top_lse)
            ids = top_id.long()
            far = (top_logit.double() * top_scale)[there].abs()
            far = float(far.max()) if len(far) else 0.0
            if top_lse is not None:
                far = max(far, float(top_lse.abs().max()))
            p_err = STEP * (4 * far + ids.shape[1] + 16)  # relative
        self.bad = (there & (ids >= v)).any(1)
        self.keep = there.any(1) & ~self.bad
        self.ids, self.p, self.p_err, self.there = torch.where(there & (ids < v), ids, 0), p, p_err, there
        # rows that do not count may hold anything
        h = torch.where(self.keep[:, None], h, 0.0)
        self.h, self.w, self.scale, self.io = h, w, scale, io
        s = scale * (h @ w.t())
        s_err = _chain(h.shape[1], io) * abs(scale) * (h.abs() @ w.abs().t()) + 3 * STEP * s.abs()
        lse = torch.logsumexp(s, 1)
        worst = s_err.amax(1)
        self.s, self.s_err, self.lse = s, s_err, lse
        size = s.abs().amax(1)
        # the exponentials' arguments, about 64 additions and a logarithm
        self.lse_err = worst + STEP * (80 + 6 * size)
        mine, mine_err = s.gather(1, self.ids), s_err.gather(1, self.ids)
        self.logq = torch.where(there, mine - lse[:, None], 0.0)
        self.logq_err = self.lse_err[:, None] + mine_err + STEP * (8 + 4 * size)[:, None]
        logp = torch.where(p > 0, torch.log(torch.where(p > 0, p, 1.0)), 0.0)
        each = torch.where(there, logp - self.logq, 0.0)
        self.loss = (p * each).sum(1)
        extra = p_err if target is None else 0.0
        self.loss_err = (p * (self.logq_err + extra + STEP * 8 * (1 + each.abs()))).sum(1) + \
            (p * each.abs()).sum(1) * extra

    def _rows(self, t):
        """The rows that are left out are 0, those with a bad id NaN."""
        shape = (-1,) + (1,) * (t.dim() - 1)
        t = torch.where(self.keep.view(shape), t, 0.0)
        return torch.where(self.bad.view(shape), float("nan"), t)

    def forward(self):
        return {"loss": (self._rows(self.loss), self.loss_err), "lse": (self._rows(self.lse), self.lse_err),
                "logq": (self._rows(self.logq), self.logq_err)}

    def backward(self, d_loss, d_lse=None, dw="f32", d_w0=None):
        keep = self.keep.double()
        d = torch.where(self.keep, d_loss.double(), 0.0) * self.scale
        dl = torch.zeros_like(d) if d_lse is None else torch.where(self.keep, d_lse.double(), 0.0) * self.scale
        mass = self.p.sum(1)
        a = d * mass + dl
        q = torch.exp(self.s - self.lse[:, None]) * keep[:, None]
        p = torch.zeros_like(q).scatter_add_(1, self.ids, torch.where(self.keep[:, None] & self.there, self.p, 0.0))
        g = a[:, None] * q - d[:, None] * p
        size = self.s.abs().amax(1, keepdim=True)
        a_err = d.abs() * mass * self.p_err + STEP * 4 * (d.abs() * mass + dl.abs())
        g_err = q * (a.abs()[:, None] * (self.s_err + self.logq_err.amax(1, keepdim=True) + STEP * (16 + 8 * size)) +
                     a_err[:, None])
        g_err = g_err + d.abs()[:, None] * p * (self.p_err + 8 * STEP)
        g_err = g_err + (HALF[self.io] if self.io == "bf16" else STEP) * (g.abs() + g_err)
        g_err = g_err + TINY * (a.abs()[:, None] + 1)
        mag = g.abs() + g_err
        dh, dh_mag = g @ self.w, mag @ self.w.abs()
        dh_err = g_err @ self.w.abs() + _chain(g.shape[1], self.io) * dh_mag + g.shape[1] * TINY
        d_w, dw_mag = g.t() @ self.h, mag.t() @ self.h.abs()
        dw_err = g_err.t() @ self.h.abs() + _chain(g.shape[0], self.io) * dw_mag + g.shape[0] * TINY
        if d_w0 is not None:
            d_w = d_w + d_w0.double()
            dw_err = dw_err + STEP * d_w.abs()
        return {"d_h": (self._rows(dh), dh_err + HALF[self.io] * (dh.abs() + dh_err)),
                "d_w": (d_w, dw_err + HALF[dw] * (d_w.abs() + dw_err))}


def check(what, got, want, err):
    want, err = want.cpu(), err.cpu()
    got = got.detach().double().cpu().reshape(want.shape)
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: NaN in other places"
    off = torch.where(want.isnan(), 0.0, (got - want).abs() - err.expand_as(want))
    if not bool((off <= 0).all()):
        at = int(torch.nan_to_num(off, nan=float("inf")).argmax())
        raise AssertionError(f"{what}: {int((~(off <= 0)).sum())} of {off.numel()} outside; worst at {at}: got "
                             f"{got.flatten()[at]!r}, want {want.flatten()[at]!r}, may be "
                             f"{err.expand_as(want).flatten()[at]!r} off")


def problem(seed, n, d, v, io, top=0, out=0.0, spread=2.5):
    """Seeded inputs on the CPU: h, w in io's type; target, or top_id and
    top_logit; d_loss."""
    gen = torch.Generator().manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen)

    w = randn(v, d) * (spread / d ** 0.5)
    first = torch.randint(v, (n,), generator=gen)
    h = randn(n, d) + torch.rand(n, 1, generator=gen) * w[first]
    t = {"h": h.to(DTYPES[io]), "w": w.to(DTYPES[io]), "d_loss": (0.5 + torch.rand(n, generator=gen)) / max(n, 1)}
    keep = torch.rand(n, generator=gen) >= out
    if top:
        ids = torch.randint(v, (n, top), generator=gen)
        ids[:, 0] = first
        there = (torch.rand(n, 1, generator=gen) > 0.2) | (torch.arange(top) < 1 + top // 2)
        t["top_id"] = torch.where(there & keep[:, None], ids, -1).int()
        t["top_logit"] = 6.0 - 1.5 * torch.log1p(torch.arange(top).float()) + 0.5 * randn(n, top)
    else:
        t["target"] = torch.where(keep, first, -100).int()
    return t
