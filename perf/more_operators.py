"""The loss over a vocabulary, as measured cases: softmax cross entropy of the
last projection's output against target tokens, and distillation from a
teacher's top logits, each as a forward pass and as a training step (forward
and backward).  The logits [rows][vocab] are never kept.

With ``own`` false run() computes them with elementary torch operations in 32
bits; with ``own`` true it calls the framework.

    s = scale * h W^T                      logits, h [rows][width], W [vocab][width]
    lse = log sum_v exp(s_v)
    cross entropy:  loss = lse - s_target; rows with a target < 0 are left out
    distillation:   p = softmax(top_scale * top_logit) over the row's entries, or
                    exp(top_scale * top_logit - top_lse) as they stand;
                    loss = sum_k p_k (log p_k - (s_id_k - lse)); entries with an
                    id < 0 are left out, and so are rows that have no other

The gradients are those of sum_i d_loss_i loss_i, in the type of h and of W.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def _case(kind, rows, width, vocab, io="bf16", top=0, out=0.0, scale=1.0, top_scale=1.0,
          as_they_stand=False, pad=0):
    return {"kind": kind, "rows": rows, "width": width, "vocab": vocab, "io": io, "top": top,
            "out": out, "scale": scale, "top_scale": top_scale, "as_they_stand": as_they_stand,
            "pad": pad}


def listed():
    # 2560 is the model width that expands to the 5120 channels of the
    # framework's scan workloads, 512 the width of its block example; 4 x 4096
    # tokens are its training batch
    return [
        # the log-probability of one decoded token: latency, W's bytes
        dict(_case("ce", 1, 2560, 32000), name="one token"),
        # a decode batch of 256 sequences is scored
        dict(_case("ce", 256, 2560, 65536), name="decode batch"),
        # the perplexity of a batch of prompts
        dict(_case("ce", 16384, 2560, 32768), name="prompts"),
        # a training step of the small block example
        dict(_case("ce_step", 512, 512, 4096), name="step, small"),
        # a training step of the large model
        dict(_case("ce_step", 16384, 2560, 32768), name="step"),
        # fine-tuning on answers: 60 of 100 tokens are prompt or padding and
        # have no target; an odd vocabulary
        dict(_case("ce_step", 8192, 2560, 50001, out=0.6), name="step, answers only"),
        # f32 at an odd size
        dict(_case("ce_step", 1023, 771, 10007, io="f32", out=0.1, pad=1), name="step, f32 odd"),
        # the distance to a teacher over a small evaluation batch
        dict(_case("kd", 64, 2560, 32000, top=16), name="teacher, evaluation"),
        # distillation of the large model from 32 logits a token
        dict(_case("kd_step", 8192, 2560, 32768, top=32, out=0.05), name="teacher step"),
        # a large vocabulary, temperature 2, the teacher's whole mass known
        dict(_case("kd_step", 2048, 2560, 131072, top=64, scale=0.5, top_scale=0.5,
                   as_they_stand=True), name="teacher step, large vocabulary"),
        # f32 at an odd size
        dict(_case("kd_step", 333, 515, 5003, io="f32", top=7, out=0.1, scale=0.7), name="teacher step, f32 odd"),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["ce", "ce_step", "kd", "kd_step"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    # widths and vocabularies of whole pieces as real models have, and odd ones
    unit = rng.choice([64, 64, 8, 1])
    width = unit * max(1, _spread(rng, 64, 5120) // unit)
    unit = rng.choice([256, 16, 1])
    vocab = unit * max(1, _spread(rng, 1000, 131072) // unit)
    most = min(16384 * 2560 * 32768 // width, 16384 * 32768) // vocab // (8 if io == "f32" else 1)
    rows = _spread(rng, 1, max(1, min(16384, most)))
    top = _spread(rng, 1, 64) if kind.startswith("kd") else 0
    return _case(kind, rows, width, vocab, io=io, top=top, out=rng.choice([0.0, 0.0, 0.1, 0.6]),
                 scale=rng.choice([1.0, 1.0, 0.5]), top_scale=rng.choice([1.0, 0.5]) if top else 1.0,
                 as_they_stand=top > 0 and rng.random() < 0.3, pad=rng.choice([0, 0, 0, 64, 3]))


def _kept(case):
    """How many rows have a target: at least one."""
    return max(1, case["rows"] - int(case["rows"] * case["out"]))


# ---- inputs ---------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    n, width, vocab, top, pad = case["rows"], case["width"], case["vocab"], case["top"], case["pad"]
    io = DTYPES[case["io"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    def padded(t):
        full = torch.zeros(t.shape[0], width + pad, dtype=io, device="cuda")
        full[:, :width] = t.to(io)
        return full[:, :width]

    s = {"case": case}
    weight = randn(vocab, width) * (2.5 / math.sqrt(width))
    first = torch.randint(vocab, (n,), generator=gen, device="cuda")
    # a normed output that knows some of its targets: their logits are raised
    # by 0 to 6
    s["h"] = padded(randn(n, width) + rand(n, 1) * weight[first])
    s["w"] = padded(weight)
    keep = torch.zeros(n, dtype=torch.bool, device="cuda")
    keep[torch.randperm(n, generator=gen, device="cuda")[:_kept(case)]] = True
    if top:
        ids = torch.randint(vocab, (n, top), generator=gen, device="cuda")
        ids[:, 0] = first
        rank = torch.arange(top, device="cuda")
        logit = 9.0 - 1.6 * torch.log1p(rank.float()) + 0.3 * randn(n, top)
        # every tenth row or so holds fewer entries
        some = (rand(n, 1) > 0.1) | (rank < 1 + int(0.6 * top))
        s["top_id"] = torch.where(some & keep[:, None], ids, -1).to(torch.int32)
        s["top_logit"] = logit
        s["top_lse"] = None
        if case["as_they_stand"]:
            # the entries hold 70 to 99 of 100 of the teacher's mass
            held = torch.logsumexp(case["top_scale"] * logit, 1)
            s["top_lse"] = held - torch.log(0.7 + 0.29 * rand(n))
    else:
        s["target"] = torch.where(keep, first, -100).to(torch.int32)
    if case["kind"].endswith("step"):
        # the mean over the rows that count, rows weighted unlike
        s["d_loss"] = (0.5 + rand(n)) / _kept(case)
    if own:
        s.update(_plan(case))
    return s


def _plan(case):
    """What a user's program keeps beside its inputs: the descriptor, the
    workspace and the output tensors."""
    from selective_scan_recurrence_amd import ops
    n, width, vocab, pad = case["rows"], case["width"], case["vocab"], case["pad"]
    io, step = DTYPES[case["io"]], case["kind"].endswith("step")
    desc = ops.vocab_desc(n_rows=n, width=width, n_vocab=vocab, n_top=case["top"], io=case["io"],
                          dw=case["io"], scale=case["scale"], top_scale=case["top_scale"],
                          ld_h=width + pad, ld_w=width + pad)
    p = {"desc": desc, "ws": ops.vocab_workspace(desc, step), "loss": torch.empty(n, device="cuda"),
         "lse": torch.empty(n, device="cuda")}
    if case["top"]:
        p["logq"] = torch.empty(n, case["top"], device="cuda")
    if step:
        p["d_h"] = torch.zeros(n, width + pad, dtype=io, device="cuda")[:, :width]
        p["d_w"] = torch.zeros(vocab, width + pad, dtype=io, device="cuda")[:, :width]
    return p


# ---- the framework's calls ---------------------------------------------------

def _run_own(s):
    from selective_scan_recurrence_amd import ops
    case = s["case"]
    step = case["kind"].endswith("step")
    if case["top"]:
        ops.vocab_kd_fwd(s["desc"], s["h"], s["w"], s["top_id"], s["top_logit"], top_lse=s["top_lse"],
                         loss=s["loss"], lse=s["lse"], logq=s["logq"], ws=s["ws"])
        if step:
            ops.vocab_kd_bwd(s["desc"], s["h"], s["w"], s["top_id"], s["top_logit"], s["logq"], s["lse"],
                             s["d_loss"], top_lse=s["top_lse"], d_h=s["d_h"], d_w=s["d_w"], ws=s["ws"])
    else:
        ops.vocab_ce_fwd(s["desc"], s["h"], s["w"], s["target"], loss=s["loss"], lse=s["lse"], ws=s["ws"])
        if step:
            ops.vocab_ce_bwd(s["desc"], s["h"], s["w"], s["target"], s["loss"], s["lse"], s["d_loss"],
                             d_h=s["d_h"], d_w=s["d_w"], ws=s["ws"])
    if step:
        return {"loss": s["loss"], "d_h": s["d_h"], "d_w": s["d_w"]}
    return {"loss": s["loss"], "lse": s["lse"]}


# ---- the plain form -------------------------------------------------------------

def _run_plain(s):
    case = s["case"]
    h, w = s["h"].float(), s["w"].float()
    logits = case["scale"] * (h @ w.t())
    top = logits.amax(1, keepdim=True)
    lse = (top + (logits - top).exp().sum(1, keepdim=True).log())
    if case["top"]:
        ids, there = s["top_id"].long().clamp(min=0), s["top_id"] >= 0
        keep = there.any(1)
        t = torch.where(there, case["top_scale"] * s["top_logit"], -math.inf)
        if s["top_lse"] is None:
            high = torch.where(keep[:, None], t.amax(1, keepdim=True), 0.0)
            mass = (t - high).exp().sum(1, keepdim=True)
            logp = t - high - torch.where(keep[:, None], mass, 1.0).log()
        else:
            logp = t - s["top_lse"][:, None]
        p = logp.exp()
        logq = logits.gather(1, ids) - lse
        loss = torch.where(there, p * (logp - logq), 0.0).sum(1)
    else:
        ids, keep = s["target"].long().clamp(min=0)[:, None], s["target"] >= 0
        p = keep[:, None].float()
        loss = torch.where(keep, (lse - logits.gather(1, ids))[:, 0], 0.0)
    if not case["kind"].endswith("step"):
        return {"loss": loss, "lse": torch.where(keep, lse[:, 0], 0.0)}
    g = logits.sub_(lse).exp_().mul_(p.sum(1, keepdim=True))
    g.scatter_add_(1, ids, -p)
    g.mul_((case["scale"] * s["d_loss"])[:, None])
    return {"loss": loss, "d_h": (g @ w).to(s["h"].dtype), "d_w": (g.t() @ h).to(s["w"].dtype)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ---------------------------------------------------

def work(case):
    n, width, vocab, top, io = _kept(case), case["width"], case["vocab"], case["top"], SIZE[case["io"]]
    step = case["kind"].endswith("step")
    data = (n + vocab) * width * io
    beside = case["rows"] * (8 + 8 * top if top else 8) + 4 * case["rows"]
    # a step: the logits, and a product for each gradient
    return {"bytes": data * (2 if step else 1) + beside + (4 * case["rows"] if step else 0),
            "flops": 2 * n * width * vocab * (3 if step else 1)}


# ---- the definition in 64 bits -----------------------------------------------------

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    n, vocab = case["rows"], case["vocab"]
    h, w = s["h"].double().contiguous(), s["w"].double().contiguous()
    step = case["kind"].endswith("step")
    loss, lse = torch.zeros(n, dtype=torch.float64, device="cuda"), torch.zeros(n, dtype=torch.float64, device="cuda")
    d_h, d_w = torch.zeros_like(h), torch.zeros_like(w)
    if case["top"]:
        ids = s["top_id"].long()
        weight = torch.exp(case["top_scale"] * s["top_logit"].double()) * (ids >= 0)
        whole = torch.exp(s["top_lse"].double()) if s["top_lse"] is not None else weight.sum(1)
        prob = weight / torch.where(whole > 0, whole, 1.0)[:, None]
    else:
        ids = s["target"].long()[:, None]
        prob = (ids >= 0).double()
    at = torch.where(ids >= 0, ids, 0)
    # a block of rows at a time: 64-bit logits of all rows take too much memory
    for rows in torch.arange(n, device="cuda").split(max(1, (1 << 28) // vocab)):
        rows = rows[(ids[rows] >= 0).any(1)]
        if not len(rows):
            continue
        x = h[rows]
        logq = torch.log_softmax(torch.mm(x, w.t().contiguous()) * case["scale"], 1)
        p, where = prob[rows], at[rows]
        mine = logq.gather(1, where)
        loss[rows] = (torch.special.xlogy(p, p) - p * mine).sum(1)
        first = where[:, 0]
        lse[rows] = (x * w[first]).sum(1) * case["scale"] - logq.gather(1, first[:, None])[:, 0]
        if step:
            wanted = torch.zeros_like(logq).scatter_add_(1, where, p)
            g = (logq.exp_() * p.sum(1, keepdim=True) - wanted) * (s["d_loss"][rows].double() * case["scale"])[:, None]
            d_h[rows] = torch.mm(g, w)
            d_w += torch.mm(g.t().contiguous(), x)
    return {"loss": loss, "d_h": d_h, "d_w": d_w} if step else {"loss": loss, "lse": lse}
