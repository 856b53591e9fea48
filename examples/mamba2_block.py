"""A stack of Mamba-2 blocks trained with 8-bit activation checkpoints, and run
token by token, on the framework's operators.

A block is norm -> projection -> selective scan -> gated norm -> projection,
added to the residual stream r:

    h = norm(r)                          norm_residual_fwd (adds the previous block's output)
    z, x, B, C, dt = h W_in^T
    y = scan(x, softplus(dt), A, B, C)   scan_fwd
    b = gated_norm(y, z) W_out^T         norm_gated_fwd

What a block keeps for its backward is 8 bits a value: r and h, x, B and C, y
and z, and the gated norm's output.  The norms write their checkpoints as they
run and their backwards read them; the scan's operands are packed and unpacked;
the projections' weight gradients are formed from the checkpoints of their
inputs.  Only dt, which sits in an exponent, is kept as it is.

    python examples/mamba2_block.py [steps]
"""
import os
import sys
from dataclasses import dataclass

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from selective_scan_recurrence_amd import ops  # noqa: E402


@dataclass
class Sizes:
    d_model: int = 512
    n_head: int = 16
    head_dim: int = 64
    d_state: int = 64
    norm_groups: int = 2
    io: str = "bf16"

    @property
    def d_inner(self):
        return self.n_head * self.head_dim

    @property
    def widths(self):
        """Of z, x, B, C, dt in the projection's output."""
        return [self.d_inner, self.d_inner, self.d_state, self.d_state, self.n_head]

    @property
    def dtype(self):
        return ops.TORCH_IO[ops.IO_DTYPES[self.io]]


def make_block(sz: Sizes, seed: int, device="cuda") -> dict:
    """Weights of a block, f32 masters."""
    gen = torch.Generator().manual_seed(seed)

    def randn(*shape, std):
        return (torch.randn(*shape, generator=gen) * std).to(device)

    return {"norm": torch.ones(sz.d_model, device=device),
            "W_in": randn(sum(sz.widths), sz.d_model, std=sz.d_model ** -0.5),
            "A": -(0.5 + torch.rand(sz.n_head, generator=gen)).to(device),
            "D": torch.ones(sz.n_head, device=device),
            "gated": torch.ones(sz.d_inner, device=device),
            "W_out": randn(sz.d_model, sz.d_inner, std=0.5 * sz.d_inner ** -0.5)}


class Stack:
    """Blocks over n_seqs sequences of n_tokens tokens."""

    def __init__(self, sz: Sizes, blocks: list, n_seqs: int, n_tokens: int, device="cuda"):
        self.sz, self.blocks = sz, blocks
        self.n_seqs, self.n_tokens, self.rows = n_seqs, n_tokens, n_seqs * n_tokens
        self.norm_out = torch.ones(sz.d_model, device=device)
        width = sum(sz.widths)
        self.scan = ops.make_desc(n_seqs=n_seqs, n_tokens=n_tokens, n_head=sz.n_head,
                                  head_dim=sz.head_dim, d_state=sz.d_state, a_per_state=False,
                                  io=sz.io, dt_softplus=True)
        self.norm = ops.norm_desc(n_rows=self.rows, width=sz.d_model, io=sz.io)
        self.gated = ops.norm_desc(n_rows=self.rows, width=sz.d_inner, n_group=sz.norm_groups,
                                   io=sz.io, ld_z=width)
        self.ids = torch.arange(n_seqs, dtype=torch.int32, device=device)
        self.state0 = torch.zeros(n_seqs, sz.n_head, sz.head_dim, sz.d_state, device=device)

    def _split(self, zxbcdt):
        sz, S, L = self.sz, self.n_seqs, self.n_tokens
        z, x, B, C, dt = zxbcdt.split(sz.widths, dim=1)
        return (z, x.contiguous().view(S, L, sz.n_head, sz.head_dim), B.contiguous().view(S, L, 1, -1),
                C.contiguous().view(S, L, 1, -1), dt.contiguous().view(S, L, sz.n_head))

    def forward(self, r, train=True):
        """The residual stream r [rows][d_model] f32 through the blocks; the
        normed output, the stream, the blocks' final scan states, and what the
        backward needs."""
        dt_, saved, states, b = self.sz.dtype, [], [], None
        for w in self.blocks:
            n = ops.norm_residual_fwd(self.norm, b, r, w["norm"], train=train)
            zxbcdt = n.h @ w["W_in"].to(dt_).t()
            z, x, B, C, dt = self._split(zxbcdt)
            scan = ops.scan_fwd(self.scan, self.state0, x, dt, w["A"], B, C, w["D"], self.ids)
            y = scan.y.view(self.rows, -1)
            out8 = ops.ckpt8_empty(self.rows, self.sz.d_inner, r.device) if train else None
            g = ops.norm_gated_fwd(self.gated, y, z, w["gated"], train=train, out8=out8)
            if train:
                packed = [ops.ckpt8_pack(t.view(self.rows, -1)) for t in (x, B, C)]
                saved.append((n.rstd, n.r8, n.h8, packed, dt, g.rstd, g.y8, g.z8, g.out8))
            states.append(scan.state)
            b, r = g.out @ w["W_out"].to(dt_).t(), n.r_out
        last = ops.norm_residual_fwd(self.norm, b, r, self.norm_out, train=train)
        return last.h, last.r_out, states, (saved, last.rstd, last.r8)

    def backward(self, dh, kept):
        """Gradients of the blocks' weights from dh, the gradient of the output."""
        sz, dt_ = self.sz, self.sz.dtype
        saved, rstd, r8 = kept
        grads = []
        last = ops.norm_residual_bwd(self.norm, dh, self.norm_out, rstd, r8=r8)
        d_r, d_b = last.d_r, last.d_b
        for w, s in zip(reversed(self.blocks), reversed(saved)):
            rstd, r8, h8, (x8, B8, C8), dt, g_rstd, y8, z8, out8 = s
            dW_out = ops.ckpt8_wgrad(d_b, out8, sz.d_inner)
            dg = d_b @ w["W_out"].to(dt_)
            # the scan's upstream gradient holds d_y, then the final state's (zero)
            dout = torch.zeros(ops.B.ssm_scan_out_bytes(self.scan), dtype=torch.uint8, device=dg.device)
            d_y, _ = ops.split_out(self.scan, dout)
            d_zxbcdt = torch.empty(self.rows, sum(sz.widths), dtype=dt_, device=dg.device)
            d_z, *d_scan = d_zxbcdt.split(sz.widths, dim=1)
            gg = ops.norm_gated_bwd(self.gated, dg, w["gated"], g_rstd, y8=y8, z8=z8,
                                    d_y=d_y.view(self.rows, -1), d_z=d_z)
            x, B, C = (ops.ckpt8_unpack(c, self.rows, n, sz.io) for c, n in
                       ((x8, sz.d_inner), (B8, sz.d_state), (C8, sz.d_state)))
            _, gs = ops.scan_bwd(self.scan, self.state0, x, dt, w["A"], B, C, w["D"], self.ids, dout)
            for to, name in zip(d_scan, ("d_x", "d_B", "d_C", "d_dt")):
                to.copy_(gs[name].view(self.rows, -1))
            dW_in = ops.ckpt8_wgrad(d_zxbcdt, h8, sz.d_model)
            dh = d_zxbcdt @ w["W_in"].to(dt_)
            gn = ops.norm_residual_bwd(self.norm, dh, w["norm"], rstd, dr_out=d_r, r8=r8, d_r=d_r)
            d_b = gn.d_b
            grads.append({"norm": gn.d_w, "W_in": dW_in, "A": gs["d_A"], "D": gs["d_D"],
                          "gated": gg.d_w, "W_out": dW_out})
        return grads[::-1], d_r


class Decoder:
    """The same blocks one token at a time, from given scan states."""

    def __init__(self, stack: Stack, states: list):
        sz, n = stack.sz, stack.n_seqs
        self.stack, self.states = stack, [s.clone() for s in states]
        self.step_desc = ops.make_desc(n_seqs=n, n_tokens=1, n_head=sz.n_head, head_dim=sz.head_dim,
                                       d_state=sz.d_state, a_per_state=False, io=sz.io, dt_softplus=True)
        self.norm = ops.norm_desc(n_rows=n, width=sz.d_model, io=sz.io)
        self.gated = ops.norm_desc(n_rows=n, width=sz.d_inner, n_group=sz.norm_groups, io=sz.io,
                                   ld_z=sum(sz.widths))

    def step(self, r):
        """One token's residual stream r [n_seqs][d_model] f32 -> the normed output."""
        st, sz, b = self.stack, self.stack.sz, None
        for w, state in zip(st.blocks, self.states):
            n = ops.norm_residual_fwd(self.norm, b, r, w["norm"])
            z, x, B, C, dt = (n.h @ w["W_in"].to(sz.dtype).t()).split(sz.widths, dim=1)
            y = ops.state_update(self.step_desc, state, x.contiguous(), dt.contiguous(), w["A"],
                                 B.contiguous(), C.contiguous(), w["D"], st.ids)
            g = ops.norm_gated_fwd(self.gated, y.view(st.n_seqs, -1), z, w["gated"])
            b, r = g.out @ w["W_out"].to(sz.dtype).t(), n.r_out
        return ops.norm_residual_fwd(self.norm, b, r, st.norm_out).h


def train(steps=40, n_blocks=2, n_seqs=4, n_tokens=128, sz=None, lr=0.05, seed=0):
    """Fits the stack to a fixed random target; returns the losses and the stack."""
    sz = sz or Sizes()
    stack = Stack(sz, [make_block(sz, seed + k) for k in range(n_blocks)], n_seqs, n_tokens)
    gen = torch.Generator().manual_seed(seed + 100)
    r = torch.randn(stack.rows, sz.d_model, generator=gen).cuda()
    target = (0.5 * torch.randn(stack.rows, sz.d_model, generator=gen)).cuda()
    losses = []
    for _ in range(steps):
        out, _, _, kept = stack.forward(r)
        diff = out.float() - target
        losses.append(float(diff.square().mean()))
        grads, _ = stack.backward((2.0 / diff.numel() * diff).to(sz.dtype), kept)
        for w, g in zip(stack.blocks, grads):
            for name, v in g.items():
                # a step of a fixed size along each weight's gradient
                w[name] -= lr * v.view_as(w[name]) * (w[name].norm() / v.norm().clamp(min=1e-20))
    return losses, stack, r


if __name__ == "__main__":
    n = int(sys.argv[1]) if len(sys.argv) > 1 else 40
    losses, stack, r = train(n)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {n} steps")
    out, _, states, _ = stack.forward(r, train=False)
    token = Decoder(stack, states).step(torch.zeros(stack.n_seqs, stack.sz.d_model, device="cuda"))
    print("next token's output:", tuple(token.shape), token.dtype)
