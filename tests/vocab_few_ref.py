"""The losses over a vocabulary for up to 64 rows of bf16: how far d_W in f32 may be
off when g enters its product as two bf16 terms.

The first term leaves up to 2^(e-8) of a g in [2^e, 2^(e+1)); the second, of what is
left (below 2^(e-8), or 2^(e-8) itself, which it holds), up to 2^(e-17): 2^-17 of g.
The rest is as in vocab_ref."""
import torch

import vocab_ref as R


class TwoTerms(R.Reference):
    """Of cross entropy, bf16."""

    def factors(self, d_loss):
        """g, and what it may be off before it is rounded."""
        d = torch.where(self.keep, d_loss.double(), 0.0) * self.scale
        q = torch.exp(self.s - self.lse[:, None]) * self.keep[:, None]
        p = torch.zeros_like(q).scatter_add_(1, self.ids, self.p * self.keep[:, None])
        size = self.s.abs().amax(1, keepdim=True)
        err = q * d.abs()[:, None] * (self.s_err + self.logq_err + R.STEP * (20 + 8 * size))
        return d[:, None] * (q - p), err + d.abs()[:, None] * (p * 8 * R.STEP + R.TINY) + R.TINY

    def d_w(self, d_loss):
        g, err = self.factors(d_loss)
        err = err + 2.0 ** -17 * (g.abs() + err)
        d_w, mag = g.t() @ self.h, (g.abs() + err).t() @ self.h.abs()
        off = err.t() @ self.h.abs() + R._chain(g.shape[0], "bf16") * mag + g.shape[0] * R.TINY
        return d_w, off + R.HALF["f32"] * (d_w.abs() + off)
