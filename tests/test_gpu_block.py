"""The operators around the scan together: the training stack of
examples/mamba2_block.py against torch autograd in float64, its decoder
against the sequence, captured graphs, and other streams."""
import importlib.util
import os

import pytest
import torch

import block_ref as R
from selective_scan_recurrence_amd import ops

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("mamba2_block", os.path.join(ROOT, "examples", "mamba2_block.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


def _reference(sz, blocks, r, dh, n_seqs, n_tokens):
    """The stack's output and weight gradients by autograd in float64 on the CPU."""
    ws = [{k: v.double().cpu().requires_grad_() for k, v in w.items()} for w in blocks]
    r = r.double().cpu()

    def norm(v, w, g=1):
        u = v.view(v.shape[0], g, -1)
        return (u / torch.sqrt(u.square().mean(-1, keepdim=True) + 1e-5)).reshape(v.shape) * w

    for w in ws:
        z, x, B, C, dt = (norm(r, w["norm"]) @ w["W_in"].t()).split(sz.widths, dim=1)
        x = x.view(n_seqs, n_tokens, sz.n_head, sz.head_dim)
        B, C = (t.view(n_seqs, n_tokens, -1) for t in (B, C))
        dt = torch.nn.functional.softplus(dt).view(n_seqs, n_tokens, sz.n_head)
        h = torch.zeros(n_seqs, sz.n_head, sz.head_dim, sz.d_state, dtype=torch.float64)
        ys = []
        for t in range(n_tokens):
            a = torch.exp(dt[:, t] * w["A"])[..., None, None]
            h = a * h + (dt[:, t, :, None] * x[:, t])[..., None] * B[:, t, None, None, :]
            ys.append((h * C[:, t, None, None, :]).sum(-1) + w["D"][:, None] * x[:, t])
        y = torch.stack(ys, 1).reshape(n_seqs * n_tokens, -1)
        r = r + norm(y * torch.nn.functional.silu(z), w["gated"], sz.norm_groups) @ w["W_out"].t()
    out = norm(r, torch.ones(sz.d_model, dtype=torch.float64))
    (out * dh.double().cpu()).sum().backward()
    return out.detach(), [{k: v.grad for k, v in w.items()} for w in ws]


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_stack_against_autograd(io):
    """Outputs are as near as the type allows.  Gradients come from 8-bit
    checkpoints, whose values are off by at most 2^-4 of themselves (evenly
    spread: 2^-4 / sqrt(3) = 3.6% rms) and enter a gradient at most three deep
    a block, two blocks: under 3.6% * sqrt(6) = 9% of its norm, so its cosine
    with the exact one is over 0.99.  (The scan's own d_A and d_D, four numbers
    each that are what is left of thousands of cancelling terms, are no such
    sums; the scan's backward has its own tests.)"""
    sz = example.Sizes(d_model=96, n_head=4, head_dim=32, d_state=64, norm_groups=2, io=io)
    blocks = [example.make_block(sz, k) for k in range(2)]
    stack = example.Stack(sz, blocks, 2, 40)
    r = torch.randn(stack.rows, sz.d_model, generator=torch.Generator().manual_seed(5)).cuda()
    dh = R.draw(6, stack.rows, sz.d_model).to(sz.dtype).cuda()
    out, _, _, kept = stack.forward(r)
    grads, _ = stack.backward(dh, kept)
    want, want_grads = _reference(sz, blocks, r, dh, 2, 40)
    err = float((out.double().cpu() - want).norm() / want.norm())
    assert err < (2e-5 if io == "f32" else 3e-2), err  # bf16: ten roundings of 2^-8 on the way
    for got, ref in zip(grads, want_grads):
        for name in ("norm", "W_in", "gated", "W_out"):
            v = ref[name]
            g = got[name].double().cpu().view_as(v)
            cos = float((g * v).sum() / (g.norm() * v.norm()))
            assert cos > 0.99, (name, cos)


def test_training_lowers_the_loss():
    losses, _, _ = example.train(steps=25, n_tokens=64)
    assert losses[-1] < 0.9 * losses[0], losses


def test_decoder_continues_the_sequence():
    """A token decoded after a prompt equals the last row of the longer prompt."""
    sz = example.Sizes(d_model=64, n_head=4, head_dim=32, d_state=32, io="f32")
    blocks = [example.make_block(sz, k) for k in range(2)]
    n_seqs, n = 3, 20
    r = torch.randn(n_seqs, n + 1, sz.d_model, generator=torch.Generator().manual_seed(1)).cuda()
    whole = example.Stack(sz, blocks, n_seqs, n + 1)
    out, _, _, _ = whole.forward(r.reshape(-1, sz.d_model), train=False)
    prompt = example.Stack(sz, blocks, n_seqs, n)
    _, _, states, _ = prompt.forward(r[:, :n].reshape(-1, sz.d_model).contiguous(), train=False)
    token = example.Decoder(prompt, states).step(r[:, n].contiguous())
    want = out.view(n_seqs, n + 1, -1)[:, n]
    assert float((token - want).norm() / want.norm()) < 1e-5


def _tensors(rows=300, width=640, groups=2):
    t = {"y": R.draw(1, rows, width).bfloat16().cuda(), "z": R.draw(2, rows, width).bfloat16().cuda(),
         "dout": R.draw(3, rows, width).bfloat16().cuda(), "r": R.draw(4, rows, width).cuda(),
         "w": (1 + 0.1 * R.draw(5, width)).cuda()}
    return t, ops.norm_desc(n_rows=rows, width=width, n_group=groups), ops.norm_desc(n_rows=rows, width=width)


def _pass(t, gated, norm, ws, kw=None):
    """Every operator once, each feeding the next."""
    kw = kw or {}
    g = ops.norm_gated_fwd(gated, t["y"], t["z"], t["w"], train=True, **kw)
    n = ops.norm_residual_fwd(norm, g.out, t["r"], t["w"], train=True, **kw)
    gn = ops.norm_residual_bwd(norm, t["dout"], t["w"], n.rstd, r8=n.r8, ws=ws[0], **kw)
    gg = ops.norm_gated_bwd(gated, gn.d_b, t["w"], g.rstd, y8=g.y8, z8=g.z8, ws=ws[0], **kw)
    dw = ops.ckpt8_wgrad(t["dout"], n.h8, t["w"].numel(), ws=ws[1], **kw)
    back = ops.ckpt8_unpack(ops.ckpt8_pack(n.h, **kw), *n.h.shape, **kw)
    return [g.out, n.r_out, n.h, gn.d_r, gn.d_w, gg.d_y, gg.d_z, gg.d_w, dw, back]


def _workspaces(t, norm):
    rows, width = t["y"].shape
    return ops.norm_bwd_workspace(norm), ops.ckpt8_wgrad_workspace(rows, width, width)


def test_captured_graph():
    """A pass captured into a graph and replayed with new inputs, with eager
    work between the replays, gives the eager results bit for bit."""
    t, gated, norm = _tensors()
    ws = _workspaces(t, norm)
    _pass(t, gated, norm, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = _pass(t, gated, norm, ws)
    for k in range(4):
        for name in ("y", "z", "dout", "r"):
            t[name].copy_(R.draw(10 * k + 7, *t[name].shape).to(t[name].dtype))
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in held]
        want = _pass(t, gated, norm, _workspaces(t, norm))
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (k, i)


@pytest.mark.parametrize("given", ["object", "address"])
def test_other_stream(given):
    """Calls queued on a stream that is not the current one, their outputs and
    workspaces left to the operators."""
    t, gated, norm = _tensors()
    want = _pass(t, gated, norm, (None, None))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kw = {"stream": side if given == "object" else side.cuda_stream}
    for _ in range(3):
        got = _pass(t, gated, norm, (None, None), kw)
        torch.ones(1 << 20, device="cuda").mul_(3)  # work and memory of the current stream
        side.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), i
