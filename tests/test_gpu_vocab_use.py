"""The losses over a vocabulary as they are used: in the block example, in captured
graphs, on other streams, two at once, and at the far ends of what they take."""
import importlib.util
import os

import pytest
import torch

import vocab_ref as R
from selective_scan_recurrence_amd import ops
from test_gpu_vocab import compare, run

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("mamba2_block", os.path.join(ROOT, "examples", "mamba2_block.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


# ---- the example ------------------------------------------------------------------


def test_example_runs():
    losses, model = example.train_tokens(steps=3, n_tokens=32, n_vocab=300)
    assert len(losses) == 3 and all(v == v and 0 < v < 100 for v in losses)
    losses, _ = example.train_tokens(steps=3, n_tokens=32, n_vocab=300, seed=10, teacher=model)
    assert all(v == v and 0 <= v < 100 for v in losses)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_example_gradients(io):
    """The head's losses and gradients after a stack, and the decoder's score of one
    token, against the 64-bit reference on the stack's own output."""
    sz = example.Sizes(d_model=96, n_head=4, head_dim=32, d_state=64, norm_groups=2, io=io)
    stack = example.Stack(sz, [example.make_block(sz, k) for k in range(2)], 3, 50)
    head = example.Head(sz, 700, stack.rows, seed=4, temperature=2.0)
    gen = torch.Generator().manual_seed(3)
    h, _, states, _ = stack.forward(torch.randn(stack.rows, sz.d_model, generator=gen).cuda(), train=False)
    target = torch.randint(-200, 700, (stack.rows,), generator=gen).int()
    d_loss = torch.rand(stack.rows, generator=gen)
    loss, g = head.tokens(h, target.cuda(), d_loss.cuda())
    ref = R.Reference(h.cpu(), head.W.to(sz.dtype).cpu(), io, target=target)
    R.check("loss", loss, *ref.forward()["loss"])
    for name, (want, err) in ref.backward(d_loss).items():
        R.check(name, getattr(g, name), want, err)
    top_logit, top_id = torch.randn(stack.rows, 9, generator=gen), torch.randint(-100, 700, (stack.rows, 9), generator=gen).int()
    loss, g = head.teacher(h, top_id.cuda(), top_logit.cuda(), d_loss.cuda())
    ref = R.Reference(h.cpu(), head.W.to(sz.dtype).cpu(), io, top_id=top_id, top_logit=top_logit, scale=0.5,
                      top_scale=0.5)
    R.check("loss", loss, *ref.forward()["loss"])
    for name, (want, err) in ref.backward(d_loss).items():
        R.check(name, getattr(g, name), want, err)
    token = example.Decoder(stack, states).step(torch.randn(3, sz.d_model, generator=gen).cuda())
    one = example.Head(sz, 700, 3, seed=4)
    score = one.score(token, torch.tensor([5, -1, 699], dtype=torch.int32, device="cuda"))
    ref = R.Reference(token.cpu(), head.W.to(sz.dtype).cpu(), io, target=torch.tensor([5, -1, 699]))
    R.check("score", score, *ref.forward()["loss"])


# ---- graphs and streams ---------------------------------------------------------------


def _on_gpu(n, d, v, io, top, seed=1):
    t = R.problem(seed, n, d, v, io, top=top, out=0.3)
    return {k: x.cuda() for k, x in t.items()}


def _pass(desc, t, ws, kw=None):
    """A forward and a backward, outputs left to the operators."""
    kw = dict(kw or {}, ws=ws)
    if desc.n_top:
        a = (desc, t["h"], t["w"], t["top_id"], t["top_logit"])
        f = ops.vocab_kd_fwd(*a, **kw)
        g = ops.vocab_kd_bwd(*a, f.logq, f.lse, t["d_loss"], **kw)
    else:
        a = (desc, t["h"], t["w"], t["target"])
        f = ops.vocab_ce_fwd(*a, **kw)
        g = ops.vocab_ce_bwd(*a, f.loss, f.lse, t["d_loss"], **kw)
    return [f.loss, f.lse, g.d_h, g.d_w] + ([f.logq] if desc.n_top else [])


CASES = [(9, 100, 500, "bf16", 0), (9, 100, 500, "f32", 3), (200, 128, 700, "bf16", 5), (200, 130, 700, "f32", 0),
         (1100, 192, 2500, "bf16", 0)]


@pytest.mark.parametrize("n,d,v,io,top", CASES)
def test_captured_graph(n, d, v, io, top):
    """Replayed with new inputs, with eager work between the replays: the eager results
    bit for bit.  Rows come and go between the replays."""
    t = _on_gpu(n, d, v, io, top)
    desc = ops.vocab_desc(n_rows=n, width=d, n_vocab=v, n_top=top, io=io)
    ws = ops.vocab_workspace(desc, True)
    _pass(desc, t, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = _pass(desc, t, ws)
    for k in range(4):
        new = R.problem(30 + k, n, d, v, io, top=top, out=[0.0, 0.9, 2.0, 0.4][k])
        for name in t:
            t[name].copy_(new[name])
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in held]
        want = _pass(desc, t, ops.vocab_workspace(desc, True))
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (k, i)


def test_two_graphs_share_a_workspace():
    """Two captured passes of unlike sizes take turns on one stream and one workspace."""
    sizes = [(200, 128, 700, "bf16", 5), (50, 128, 900, "bf16", 0)]
    ts = [_on_gpu(*s) for s in sizes]
    descs = [ops.vocab_desc(n_rows=n, width=d, n_vocab=v, n_top=top, io=io) for n, d, v, io, top in sizes]
    ws = max((ops.vocab_workspace(d, True) for d in descs), key=lambda w: w.numel())
    want = [_pass(d, t, None) for d, t in zip(descs, ts)]
    torch.cuda.synchronize()
    graphs, held = [], []
    for d, t in zip(descs, ts):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(_pass(d, t, ws))
    for _ in range(3):
        for g, h in zip(graphs, held):
            for x in h:
                x.zero_()
            g.replay()
    torch.cuda.synchronize()
    for a, b in zip(held, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("given", ["object", "address"])
@pytest.mark.parametrize("n,d,v,io,top", CASES[:3])
def test_other_stream(n, d, v, io, top, given):
    """Queued on a stream that is not the current one, outputs and workspaces left to the
    operators."""
    t = _on_gpu(n, d, v, io, top)
    desc = ops.vocab_desc(n_rows=n, width=d, n_vocab=v, n_top=top, io=io)
    want = _pass(desc, t, None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kw = {"stream": side if given == "object" else side.cuda_stream}
    for _ in range(3):
        got = _pass(desc, t, None, kw)
        torch.ones(1 << 20, device="cuda").mul_(3)  # work and memory of the current stream
        side.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), i


def test_two_calls_at_once():
    """Two streams, a workspace each."""
    n, d, v = 600, 256, 3000
    ts = [_on_gpu(n, d, v, "bf16", 0, seed) for seed in (1, 2)]
    desc = ops.vocab_desc(n_rows=n, width=d, n_vocab=v)
    want = [_pass(desc, t, None) for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    wss = [ops.vocab_workspace(desc, True) for _ in ts]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        got = [_pass(desc, t, ws, {"stream": s}) for t, ws, s in zip(ts, wss, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


# ---- far ends -----------------------------------------------------------------------


@pytest.mark.parametrize("scale", [-0.7, 0.0, 3.0])
@pytest.mark.parametrize("n", [5, 140])
def test_scales(n, scale):
    t = R.problem(40, n, 96, 333, "bf16", out=0.2)
    compare(t, "bf16", run(t, "bf16", scale=scale), scale=scale)


@pytest.mark.parametrize("n", [2, 70])
def test_most_entries(n):
    t = R.problem(41, n, 64, 3000, "f32", top=1024)
    compare(t, "f32", run(t, "f32"))


@pytest.mark.parametrize("io,top", [("bf16", 0), ("bf16", 70), ("f32", 0)])
def test_big_tiles(io, top):
    """Enough rows, vocabulary and width for the 256 x 256 tiles in every product, with
    ragged ends.  The reference runs on the GPU, in 64 bits."""
    t = R.problem(42, 4090, 2042, 4001, io, top=top, out=0.02)
    on_gpu = {k: v.cuda() for k, v in t.items()}
    compare(on_gpu, io, run(t, io, dw=io), dw=io)


@pytest.mark.parametrize("n,d,v,io,top", [
    (1, 64, 40, "bf16", 0), (17, 130, 5000, "bf16", 3), (64, 65, 300, "f32", 0), (65, 65, 129, "bf16", 0),
    (300, 70, 5000, "f32", 5), (130, 200, 30000, "bf16", 0), (5000, 33, 300, "bf16", 2), (2048, 96, 2100, "f32", 0),
])
@pytest.mark.parametrize("only", ["d_h", "d_w", None])
def test_nothing_behind_the_workspace_is_written(n, d, v, io, top, only):
    t = _on_gpu(n, d, v, io, top)
    desc = ops.vocab_desc(n_rows=n, width=d, n_vocab=v, n_top=top, io=io)
    for backward in (False, True):
        size = ops.vocab_workspace(desc, backward).numel()
        whole = torch.full((size + 65536,), 0xA5, dtype=torch.uint8, device="cuda")
        ws = whole[:size]
        if top:
            f = ops.vocab_kd_fwd(desc, t["h"], t["w"], t["top_id"], t["top_logit"], ws=ws)
        else:
            f = ops.vocab_ce_fwd(desc, t["h"], t["w"], t["target"], ws=ws)
        if backward:
            kw = dict(ws=ws, want_h=only != "d_w", want_w=only != "d_h")
            if top:
                ops.vocab_kd_bwd(desc, t["h"], t["w"], t["top_id"], t["top_logit"], f.logq, f.lse, t["d_loss"], **kw)
            else:
                ops.vocab_ce_bwd(desc, t["h"], t["w"], t["target"], f.loss, f.lse, t["d_loss"], **kw)
        assert bool((whole[size:] == 0xA5).all())


@pytest.mark.parametrize("n,d,v,io", [(40, 70, 3000, "bf16"), (3000, 70, 300, "bf16"), (300, 70, 5000, "f32")])
def test_either_gradient_alone(n, d, v, io):
    """Its parts may be others than with both: the same values within the bounds."""
    t = R.problem(46, n, d, v, io, out=0.2)
    desc = ops.vocab_desc(n_rows=n, width=d, n_vocab=v, io=io)
    g = {k: x.cuda() for k, x in t.items()}
    f = ops.vocab_ce_fwd(desc, g["h"], g["w"], g["target"])
    a = (desc, g["h"], g["w"], g["target"], f.loss, f.lse, g["d_loss"])
    one, other = ops.vocab_ce_bwd(*a, want_w=False), ops.vocab_ce_bwd(*a, want_h=False)
    assert one.d_w is None and other.d_h is None
    want = R.Reference(t["h"], t["w"], io, target=t["target"]).backward(t["d_loss"])
    R.check("d_h", one.d_h, *want["d_h"])
    R.check("d_w", other.d_w, *want["d_w"])


@pytest.mark.parametrize("spread,top", [(64, 40), (5, 12), (100, 70)])
@pytest.mark.parametrize("n", [3, 70, 300])
def test_ids_close_together(n, spread, top):
    """Many ids of a row within a few neighbours of the vocabulary."""
    t = R.problem(44, n, 64, 700, "bf16", top=top)
    t["top_id"] = torch.where(t["top_id"] < 0, -1, 130 + t["top_id"] % spread).int()
    if spread < top:  # entries with the same id hold the same logit's two shares
        t["top_id"][:, spread:] = t["top_id"][:, :1]
    compare(t, "bf16", run(t, "bf16"))


@pytest.mark.parametrize("n,d,v,io,dw", [(3000, 70, 256, "bf16", "f32"), (3000, 130, 300, "bf16", "bf16"),
                                         (1100, 65, 129, "f32", "f32"), (70, 65, 9000, "f32", "f32")])
@pytest.mark.parametrize("add,out", [(False, 0.1), (True, 0.1), (False, 0.9)])
def test_long_sums_for_few_tiles(n, d, v, io, dw, add, out):
    """Sums over many rows or a long vocabulary for small gradients, formed in parts: the
    more of them the more rows are left out."""
    t = R.problem(45, n, d, v, io, out=out)
    d_w0 = None
    if add:
        d_w0 = (0.01 * torch.randn(v, d, generator=torch.Generator().manual_seed(5))).to(R.DTYPES[dw])
    compare(t, io, run(t, io, dw=dw, d_w0=d_w0, pad_w=3), dw=dw, d_w0=d_w0)


@pytest.mark.parametrize("n", [3, 130])
def test_weights_past_4_gigabytes(n):
    """W of 36000 x 65536: rows whose offset passes 32 bits.  All zero but for a value on
    each of a few rows, so that the losses are known."""
    v, d = 36000, 65536
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    rows = torch.tensor([0, 1, 16383, 32767, 32768, 32769, 35999])
    value = torch.linspace(1, 3, len(rows))
    w = torch.zeros(v, d, dtype=torch.bfloat16, device="cuda")
    w[rows, d - 1] = value.bfloat16().cuda()
    h = torch.zeros(n, d, dtype=torch.bfloat16, device="cuda")
    h[:, d - 1] = (1.0 + torch.arange(n) % 4).bfloat16().cuda()
    target = rows[torch.arange(n) % len(rows)].int()
    s = torch.zeros(n, v, dtype=torch.float64)
    s[:, rows] = (1.0 + torch.arange(n) % 4).double()[:, None] * value.bfloat16().double()
    lse = torch.logsumexp(s, 1)
    desc = ops.vocab_desc(n_rows=n, width=d, n_vocab=v, dw="bf16")
    f = ops.vocab_ce_fwd(desc, h, w, target.cuda())
    want = lse - s.gather(1, target.long()[:, None])[:, 0]
    # exact products and one addition that is not of zeros; then the statistics as in vocab_ref
    assert float((f.loss.double().cpu() - want).abs().max()) < R.STEP * (80 + 12 * 12)
    d_loss = torch.full((n,), 1.0, device="cuda")
    g = ops.vocab_ce_bwd(desc, h, w, target.cuda(), f.loss, f.lse, d_loss)
    q = torch.exp(s - lse[:, None])
    q[torch.arange(n), target.long()] -= 1.0
    want_w = (q.t() @ h[:, d - 1].double().cpu())[rows]
    got_w = g.d_w[rows, d - 1].double().cpu()
    # g's terms, the statistics' error 1e-5, and the output's rounding
    assert float((got_w - want_w).abs().max()) < 2 * R.HALF["bf16"] * float(q.abs().t().mul(4).sum(1).max())
    want_h = q[:, rows] @ value.bfloat16().double()
    assert float((g.d_h[:, d - 1].double().cpu() - want_h).abs().max()) < 3 * R.HALF["bf16"] * float(q[:, rows].abs().sum(1).max() * 3)
    assert float(g.d_h[:, :d - 1].abs().max()) == 0.0 and float(g.d_w[:, :d - 1].abs().max()) == 0.0
    del w, h, g
    torch.cuda.empty_cache()


def test_the_most_rows():
    """2^21 rows, most of them left out: lists, tensors and pieces at their longest.  Logits
    that depend on the row's and the entry's number alone, so that losses are known."""
    n, d, v = 1 << 21, 8, 300
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    gen = torch.Generator(device="cuda").manual_seed(5)
    h = torch.randn(n, d, generator=gen, device="cuda").bfloat16()
    w = torch.randn(v, d, generator=gen, device="cuda").bfloat16()
    target = torch.randint(-2 * v, v, (n,), generator=gen, device="cuda").int()
    target[-1], target[0] = 299, 0
    keep = target >= 0
    desc = ops.vocab_desc(n_rows=n, width=d, n_vocab=v)
    f = ops.vocab_ce_fwd(desc, h, w, target)
    d_loss = torch.rand(n, generator=gen, device="cuda")
    g = ops.vocab_ce_bwd(desc, h, w, target, f.loss, f.lse, d_loss)
    d_w = torch.zeros(v, d, dtype=torch.float64, device="cuda")
    mag = torch.zeros(v, d, dtype=torch.float64, device="cuda")
    for rows in torch.arange(n, device="cuda").split(1 << 18):
        s = h[rows].double() @ w.double().t()
        size = float(s.abs().max())
        lse = torch.logsumexp(s, 1)
        at = target[rows].long().clamp(min=0)
        want = torch.where(keep[rows], lse - s.gather(1, at[:, None])[:, 0], 0.0)
        # 8 exact products: 8 additions, then the statistics as in vocab_ref
        tol = R.STEP * (80 + 12 * size + 20 * float((h[rows].double().abs() @ w.double().abs().t()).max()))
        assert float((f.loss[rows].double() - want).abs().max()) < tol
        q = torch.exp(s - lse[:, None])
        q[torch.arange(len(rows), device="cuda"), at] -= 1.0
        q *= torch.where(keep[rows], d_loss[rows].double(), 0.0)[:, None]
        dh = q @ w.double()
        err = (2 * R.HALF["bf16"] + 2 * tol) * (q.abs() @ w.double().abs()) + R.HALF["bf16"] * dh.abs()
        assert bool(((g.d_h[rows].double() - dh).abs() <= err).all())
        d_w += q.t() @ h[rows].double()
        mag += q.abs().t() @ h[rows].double().abs()
    # a rounding of g each, and one addition a row at most
    assert bool(((g.d_w.double() - d_w).abs() <= (2 * R.HALF["bf16"] + 2 * tol + R.STEP * n / 8) * mag).all())
    assert bool((g.d_h[~keep] == 0).all()) and bool((f.loss[~keep] == 0).all())
    del h, w, f, g
    torch.cuda.empty_cache()
