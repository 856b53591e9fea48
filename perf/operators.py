"""The operators around the scan in a Mamba block, as measured cases: the norm
between two blocks (residual add, residual scale, norm after the block and
before the next), the gated norm after the scan, activation checkpoints in 8
bits, and the projection's weight gradient from such a checkpoint.

With ``own`` false run() computes them with elementary torch operations in 32
bits; with ``own`` true it calls the framework.

The 8-bit checkpoint of a [rows][width] tensor: along each row, blocks of 32
values share a scale 2^k, the smallest with max|x| <= 448 * 2^k, and each value
is kept as e4m3 of x / 2^k.  In memory: the codes [rows][width rounded up to
32], padded with zeros, then the scale bytes k + 127 [rows][blocks].
"""
import math

import torch

own = False

EPS = 1e-5
BLOCK = 32
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def _case(kind, rows, width, io="bf16", res="f32", ckpt=False, group=1, after=False, post=False,
          scale=False, alpha=1.0, pad=0, n_out=0):
    return {"kind": kind, "rows": rows, "width": width, "io": io, "res": res, "ckpt": ckpt,
            "group": group, "after": after, "post": post, "scale": scale, "alpha": alpha,
            "pad": pad, "n_out": n_out}


def listed():
    # 5120 channels is the layer of the framework's scan workloads, 2560 the
    # model width that expands to it, 10576 = 2 * 5120 + 2 * 128 + 80 the width
    # of the projection before the Mamba-2 form (z, x, B, C, dt)
    return [
        # one decoded token enters a block: latency
        dict(_case("residual_fwd", 1, 2560), name="residual, one token"),
        # a prompt batch of 4 x 4096 tokens, a constant residual scale
        dict(_case("residual_fwd", 16384, 2560, alpha=0.25), name="residual, prompts"),
        # training: the same batch, the backward from the 8-bit residual stream
        dict(_case("residual_step", 16384, 2560, ckpt=True), name="residual step, 8-bit"),
        # training in f32 at an odd size: norm after the block, learned residual scale
        dict(_case("residual_step", 2047, 1283, io="f32", post=True, scale=True, alpha=0.5),
             name="residual step, both norms"),
        # a decode batch of 256 sequences; z is a slice of the projection's output
        dict(_case("gated_fwd", 256, 5120, pad=5456), name="gated, decode batch"),
        # a prompt batch of 8 x 4096 tokens
        dict(_case("gated_fwd", 32768, 5120, pad=5456), name="gated, prompts"),
        # training with 8 norm groups: the backward from 8-bit y and z
        dict(_case("gated_step", 16384, 5120, ckpt=True, group=8, pad=5456), name="gated step, 8-bit"),
        # training in f32 at an odd size, the gate after the norm
        dict(_case("gated_step", 1111, 771, io="f32", group=3, after=True, pad=1), name="gated step, gate after"),
        # the scan's x kept in 8 bits for its backward and read back
        dict(_case("ckpt", 32768, 5120, pad=5456), name="checkpoint of x"),
        # a short f32 row block
        dict(_case("ckpt", 64, 515, io="f32"), name="checkpoint, short"),
        # weight gradient of the projection into the block
        dict(_case("wgrad", 8192, 2560, n_out=10576), name="weight gradient"),
        # the same in f32 for a small odd projection
        dict(_case("wgrad", 777, 515, io="f32", n_out=130), name="weight gradient, odd"),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["residual_fwd", "residual_step", "gated_fwd", "gated_step", "ckpt", "wgrad"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if kind == "wgrad":
        width, n_out = _spread(rng, 32, 5120), _spread(rng, 16, 10576)
        most = 8192 * 2560 * 10576 // (width * n_out) // (4 if io == "f32" else 1)
        return _case(kind, _spread(rng, 1, min(32768, max(1, most))), width, io=io, n_out=n_out,
                     pad=rng.choice([0, 0, 3, 16]))
    group = rng.choice([1, 1, 2, 8]) if kind.startswith("gated") else 1
    # rows of whole 16-byte pieces as real layers have, and odd ones
    unit = rng.choice([64, 32, 8, 1])
    ckpt = kind.endswith("step") and rng.random() < 0.5
    if ckpt and group > 1:
        unit = 32
    width = group * unit * max(1, _spread(rng, 64, 8192) // (group * unit))
    most = 16384 * 2560 if kind.startswith("residual") else 16384 * 5120
    rows = _spread(rng, 1, max(1, most // width // (2 if io == "f32" else 1)))
    pad = rng.choice([0, 0, 8, 64, 5])
    if kind.startswith("residual"):
        post, scale = rng.random() < 0.4, rng.random() < 0.4
        # a stream that is kept in 8 or 16 bits is a plain sum here: the same
        # whatever the order of operations, so that no rounding falls elsewhere
        if ckpt:
            post = scale = False
        alpha = 1.0 if ckpt else rng.choice([1.0, 0.25, 0.7])
        res = "f32" if post or scale or alpha == 0.7 else rng.choice(["f32", io])
        return _case(kind, rows, width, io=io, res=res, ckpt=ckpt, post=post, scale=scale,
                     alpha=alpha, pad=pad)
    if kind == "ckpt":
        return _case(kind, rows, width, io=io, pad=pad)
    return _case(kind, rows, width, io=io, ckpt=ckpt, group=group, after=rng.random() < 0.5, pad=pad)


# ---- inputs ---------------------------------------------------------------

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=gen.device)


def _activation(gen, rows, width, dtype, pad=0, loud=True):
    """[rows][width] in rows of width + pad: channels of unlike size, a few of
    them loud, as the residual stream and the scan's output have."""
    gain = torch.exp(0.5 * _randn(gen, width))
    if loud:
        gain[torch.rand(width, generator=gen, device=gen.device) < 0.004] *= 12.0
    x = torch.zeros(rows, width + pad, dtype=dtype, device=gen.device)
    x[:, :width] = (_randn(gen, rows, width) * gain).to(dtype)
    return x[:, :width]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    kind, m, w, pad = case["kind"], case["rows"], case["width"], case["pad"]
    io, res = DTYPES[case["io"]], DTYPES[case["res"]]
    s = {"case": case}
    if kind == "wgrad":
        s["dy"] = _activation(gen, m, case["n_out"], io, pad, loud=False)
        s["x8"] = _pack(_activation(gen, m, w, torch.float32))
    elif kind == "ckpt":
        s["x"] = _activation(gen, m, w, io, pad)
    elif kind.startswith("residual"):
        s["b"] = _activation(gen, m, w, io, pad)
        s["r"] = (4.0 * _activation(gen, m, w, torch.float32)).to(res)
        s["w"] = 1.0 + 0.1 * _randn(gen, w)
        s["w_post"] = 1.0 + 0.1 * _randn(gen, w) if case["post"] else None
        s["scale"] = 0.1 + 0.02 * _randn(gen, w) if case["scale"] else None
        if kind == "residual_step":
            s["dh"] = _activation(gen, m, w, io, 0, loud=False)
            s["dr_out"] = _activation(gen, m, w, res, 0, loud=False)
    else:
        s["y"] = _activation(gen, m, w, io)
        s["z"] = _activation(gen, m, w, io, pad, loud=False)
        s["w"] = 1.0 + 0.1 * _randn(gen, w)
        if kind == "gated_step":
            s["dout"] = _activation(gen, m, w, io, 0, loud=False)
    if own:
        s.update(_plan(case, s))
    return s


def _plan(case, s):
    """What a user's program keeps beside its inputs: the descriptor, the
    workspace and the output tensors."""
    from selective_scan_recurrence_amd import ops
    kind, m, w, pad = case["kind"], case["rows"], case["width"], case["pad"]
    io, res, dev = DTYPES[case["io"]], DTYPES[case["res"]], "cuda"

    def new(dtype, extra=0):
        return torch.zeros(m, w + extra, dtype=dtype, device=dev)[:, :w]

    if kind == "wgrad":
        return {"dw": torch.empty(case["n_out"], w, device=dev),
                "ws": ops.ckpt8_wgrad_workspace(m, w, case["n_out"], case["io"], dev)}
    if kind == "ckpt":
        return {"x8": ops.ckpt8_empty(m, w, dev), "back": new(io)}
    step = kind.endswith("step")
    gated = kind.startswith("gated")
    desc = ops.norm_desc(n_rows=m, width=w, n_group=case["group"], io=case["io"], res=case["res"],
                         eps=EPS, res_scale=case["alpha"], gate_after=case["after"],
                         ld_x=w if gated else w + pad, ld_z=w + pad if gated else 0)
    p = {"desc": desc}
    if step:
        p["ws"] = ops.norm_bwd_workspace(desc, dev)
        p["rstd"] = torch.empty(m, case["group"], device=dev)
        p["dw"] = torch.empty(w, device=dev)
    if gated:
        p["out"] = new(io)
        if step:
            p["dy"], p["dz"] = new(io), new(io, pad)
            p["y8"], p["z8"] = (ops.ckpt8_empty(m, w, dev) if case["ckpt"] else None for _ in range(2))
        return p
    p["r_out"], p["h"] = new(res), new(io)
    if step:
        p["rstd_post"] = torch.empty(m, device=dev) if case["post"] else None
        p["d_r"], p["d_b"] = new(res), new(io, pad)
        p["r8"] = ops.ckpt8_empty(m, w, dev) if case["ckpt"] else None
        p["d_w_post"] = torch.empty(w, device=dev) if case["post"] else None
        p["d_scale"] = torch.empty(w, device=dev) if case["scale"] else None
    return p


# ---- the framework's calls ---------------------------------------------------

def _run_own(s):
    from selective_scan_recurrence_amd import ops
    case = s["case"]
    kind = case["kind"]
    if kind == "wgrad":
        return ops.ckpt8_wgrad(s["dy"], s["x8"], case["width"], dw=s["dw"], ws=s["ws"])
    if kind == "ckpt":
        ops.ckpt8_pack(s["x"], out=s["x8"])
        return ops.ckpt8_unpack(s["x8"], case["rows"], case["width"], out=s["back"])
    if kind.startswith("gated"):
        step, ckpt = kind == "gated_step", case["ckpt"]
        ops.norm_gated_fwd(s["desc"], s["y"], s["z"], s["w"], out=s["out"], rstd=s.get("rstd"),
                           y8=s.get("y8"), z8=s.get("z8"))
        if not step:
            return s["out"]
        ops.norm_gated_bwd(s["desc"], s["dout"], s["w"], s["rstd"], y=None if ckpt else s["y"],
                           z=None if ckpt else s["z"], y8=s["y8"], z8=s["z8"], d_y=s["dy"],
                           d_z=s["dz"], d_w=s["dw"], ws=s["ws"])
        return {"out": s["out"], "d_y": s["dy"], "d_z": s["dz"], "d_w": s["dw"]}
    ops.norm_residual_fwd(s["desc"], s["b"], s["r"], s["w"], w_post=s["w_post"], scale=s["scale"],
                          r_out=s["r_out"], h=s["h"], rstd=s.get("rstd"),
                          rstd_post=s.get("rstd_post"), r8=s.get("r8"))
    if kind == "residual_fwd":
        return {"r_out": s["r_out"], "h": s["h"]}
    need_b = case["post"] or case["scale"]
    ops.norm_residual_bwd(s["desc"], s["dh"], s["w"], s["rstd"], dr_out=s["dr_out"],
                          r_out=None if case["ckpt"] else s["r_out"], r8=s["r8"],
                          b=s["b"] if need_b else None, rstd_post=s["rstd_post"],
                          w_post=s["w_post"], scale=s["scale"], d_r=s["d_r"], d_b=s["d_b"],
                          d_w=s["dw"], d_w_post=s["d_w_post"], d_scale=s["d_scale"], ws=s["ws"])
    return {"r_out": s["r_out"], "h": s["h"], "d_r": s["d_r"], "d_b": s["d_b"], "d_w": s["dw"],
            "d_w_post": s["d_w_post"], "d_scale": s["d_scale"]}


# ---- the plain form -------------------------------------------------------------

def _pow2(k):
    """2^k in f32 for whole k, without the rounding of a power function."""
    return ((k.long() + 1023) << 52).view(torch.float64).float()


def _codes(x):
    """e4m3 codes [rows][blocks][32] and exponents [rows][blocks] of x."""
    rows, width = x.shape
    blocks = -(-width // BLOCK)
    v = torch.zeros(rows, blocks * BLOCK, device=x.device)
    v[:, :width] = x.float()
    v = v.view(rows, blocks, BLOCK)
    finite = torch.isfinite(v)
    amax = torch.where(finite, v.abs(), 0.0).amax(-1)
    frac, exp = torch.frexp(amax)
    k = torch.where(amax > 0, exp - 9 + (frac > 0.875), -127).clamp(min=-127)
    scaled = torch.where(finite, v * _pow2(-k).unsqueeze(-1), math.nan)
    return scaled.to(torch.float8_e4m3fn), k


def _kept(x):
    """x as its 8-bit checkpoint keeps it, in f32."""
    codes, k = _codes(x)
    v = codes.float() * _pow2(k).unsqueeze(-1)
    return v.view(x.shape[0], -1)[:, :x.shape[1]]


def _pack(x):
    codes, k = _codes(x)
    return torch.cat([codes.view(torch.uint8).reshape(-1), (k + 127).to(torch.uint8).reshape(-1)])


def _unpack(x8, rows, width):
    blocks = -(-width // BLOCK)
    n = rows * blocks * BLOCK
    codes = x8[:n].view(torch.float8_e4m3fn).float().view(rows, blocks, BLOCK)
    k = x8[n:].long().view(rows, blocks, 1) - 127
    return (codes * _pow2(k)).view(rows, -1)[:, :width]


def _rstd(x):
    return torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _norm_grad(dn, xhat, rstd):
    return rstd * (dn - xhat * (dn * xhat).mean(-1, keepdim=True))


def _run_plain(s):
    case = s["case"]
    kind, m, w = case["kind"], case["rows"], case["width"]
    io, res = DTYPES[case["io"]], DTYPES[case["res"]]
    if kind == "wgrad":
        return s["dy"].float().t() @ _unpack(s["x8"], m, w)
    if kind == "ckpt":
        return _kept(s["x"]).to(io)
    if kind.startswith("gated"):
        split = (m, case["group"], -1)
        y, z, wt = s["y"].float().view(split), s["z"].float().reshape(split), s["w"].view(case["group"], -1)
        g = z * torch.sigmoid(z)
        u = y if case["after"] else y * g
        rstd = _rstd(u)
        n = u * rstd * wt
        out = ((n * g) if case["after"] else n).view(m, w).to(io)
        if kind == "gated_fwd":
            return out
        if case["ckpt"]:
            y, z = _kept(s["y"]).reshape(split), _kept(s["z"]).reshape(split)
        sg = torch.sigmoid(z)
        g, slope = z * sg, sg * (1.0 + z * (1.0 - sg))
        dout = s["dout"].float().view(split)
        if case["after"]:
            xhat = y * rstd
            dz = dout * xhat * wt * slope
            dw = (dout * g * xhat).sum(0)
            dy = _norm_grad(dout * g * wt, xhat, rstd)
        else:
            xhat = y * g * rstd
            dw = (dout * xhat).sum(0)
            du = _norm_grad(dout * wt, xhat, rstd)
            dy, dz = du * g, du * y * slope
        return {"out": out, "d_y": dy.view(m, w).to(io), "d_z": dz.view(m, w).to(io), "d_w": dw.view(w)}
    b, r = s["b"].float(), s["r"].float()
    gain = case["alpha"] if s["scale"] is None else case["alpha"] * s["scale"]
    t = b
    if case["post"]:
        rstd_post = _rstd(b)
        t = b * rstd_post * s["w_post"]
    x = r + gain * t
    rstd = _rstd(x)
    r_out, h = x.to(res), (x * rstd * s["w"]).to(io)
    if kind == "residual_fwd":
        return {"r_out": r_out, "h": h}
    xhat = (_kept(r_out) if case["ckpt"] else r_out.float()) * rstd
    dh = s["dh"].float()
    dx = _norm_grad(dh * s["w"], xhat, rstd) + s["dr_out"].float()
    dt = gain * dx
    d_w_post = None
    if case["post"]:
        bhat = b * rstd_post
        d_w_post = (dt * bhat).sum(0)
        d_b = _norm_grad(dt * s["w_post"], bhat, rstd_post)
    else:
        d_b = dt
    d_scale = (case["alpha"] * dx * t).sum(0) if case["scale"] else None
    return {"r_out": r_out, "h": h, "d_r": dx.to(res), "d_b": d_b.to(io), "d_w": (dh * xhat).sum(0),
            "d_w_post": d_w_post, "d_scale": d_scale}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ---------------------------------------------------

def work(case):
    kind, m, w = case["kind"], case["rows"], case["width"]
    io, res, n = SIZE[case["io"]], SIZE[case["res"]], m * w
    kept = m * (-(-w // BLOCK)) * (BLOCK + 1)
    if kind == "wgrad":
        o = case["n_out"]
        return {"bytes": m * o * io + kept + 4 * o * w, "flops": 2 * m * w * o}
    if kind == "ckpt":  # pack, then unpack
        return {"bytes": 2 * (n * io + kept), "flops": 4 * n}
    if kind.startswith("gated"):
        total, flops = n * 3 * io + 4 * w, 10 * n
        if kind == "gated_step":
            total += n * 3 * io + 8 * w + 8 * m * case["group"]
            total += 4 * kept if case["ckpt"] else 2 * n * io
            flops += 20 * n
        return {"bytes": total, "flops": flops}
    total, flops = n * 2 * (io + res) + 4 * w * (1 + case["post"] + case["scale"]), 6 * n
    if kind == "residual_step":
        total += n * 2 * (io + res) + 8 * m * (1 + case["post"]) + 8 * w * (1 + case["post"] + case["scale"])
        total += 2 * kept if case["ckpt"] else n * res
        total += n * io if case["post"] or case["scale"] else 0
        flops += 14 * n
    return {"bytes": total, "flops": flops}


# ---- the definition in 64 bits -----------------------------------------------------

def _kept64(x):
    """The checkpoint's values in 64 bits, from its definition: the e4m3 grid
    has steps of 2^(e - 3) in [2^e, 2^(e + 1)), down to e = -6."""
    def two(k):  # 2^k, k whole, built by its bits: a power function rounds
        return ((k.to(torch.int64) + 1023) * 2 ** 52).view(torch.float64)

    rows, width = x.shape
    short = -width % BLOCK
    v = torch.nn.functional.pad(x.double(), (0, short)).unflatten(1, (-1, BLOCK))
    top = v.abs().amax(-1, keepdim=True)
    k = torch.ceil(torch.log2(torch.clamp(top, min=2.0 ** -150) / 448.0))
    # the logarithm may be a step off at a border
    k = torch.where(top > 448.0 * two(k), k + 1, k)
    k = torch.where(top <= 448.0 * two(k - 1), k - 1, k).clamp(min=-127)
    v = v / two(k)
    e = torch.floor(torch.log2(torch.clamp(v.abs(), min=2.0 ** -6)))
    e = torch.where(v.abs() >= two(e + 1), e + 1, e)
    e = torch.where(v.abs() < two(e), e - 1, e).clamp(min=-6)
    step = two(e - 3)
    return (torch.round(v / step) * step * two(k)).flatten(1)[:, :width]


def _unpack64(x8, rows, width):
    """The codes read bit by bit: sign, four exponent bits (bias 7), three mantissa bits."""
    blocks = -(-width // BLOCK)
    c = x8[:rows * blocks * BLOCK].long().view(rows, blocks, BLOCK)
    k = x8[rows * blocks * BLOCK:].long().view(rows, blocks, 1) - 127
    e, f = (c >> 3) & 15, c & 7
    whole = torch.where(e == 0, f, 8 + f) << torch.clamp(e - 1, min=0)  # in steps of 2^-9
    mag = whole.double() * ((k - 9 + 1023) * 2 ** 52).view(torch.float64)
    return torch.where(c >= 128, -mag, mag).flatten(1)[:, :width]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    kind, m, w, groups = case["kind"], case["rows"], case["width"], case["group"]
    if kind == "wgrad":
        return torch.mm(s["dy"].double().t().contiguous(), _unpack64(s["x8"], m, w))
    if kind == "ckpt":
        return _kept64(s["x"])
    p = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}

    def grouped(v):
        return v.reshape(m, groups, w // groups)

    def norm(v):  # (v / rms, 1 / rms)
        inv = 1.0 / torch.sqrt((grouped(v) ** 2).sum(-1, keepdim=True) * (groups / w) + EPS)
        return (grouped(v) * inv).reshape(m, w), inv

    def norm_back(d, unit, inv):
        c = (grouped(d) * grouped(unit)).sum(-1, keepdim=True) * (groups / w)
        return ((grouped(d) - grouped(unit) * c) * inv).reshape(m, w)

    if kind.startswith("gated"):
        y, z = p["y"], p["z"]
        silu = z / (1.0 + torch.exp(-z))
        unit, inv = norm(y if case["after"] else y * silu)
        out = unit * p["w"] * (silu if case["after"] else 1.0)
        if kind == "gated_fwd":
            return out
        if case["ckpt"]:
            y, z = _kept64(s["y"]), _kept64(s["z"])
        silu = z / (1.0 + torch.exp(-z))
        # d SiLU / dz = SiLU(z) + sigmoid(z) (1 - SiLU(z))
        slope = silu + (1.0 - silu) / (1.0 + torch.exp(-z))
        unit = (grouped(y if case["after"] else y * silu) * inv).reshape(m, w)
        d = p["dout"]
        if case["after"]:
            d_n = d * silu
            d_z = d * unit * p["w"] * slope
            d_y = norm_back(d_n * p["w"], unit, inv)
            d_w = (d_n * unit).sum(0)
        else:
            d_u = norm_back(d * p["w"], unit, inv)
            d_y, d_z, d_w = d_u * silu, d_u * y * slope, (d * unit).sum(0)
        return {"out": out, "d_y": d_y, "d_z": d_z, "d_w": d_w}
    t, b_unit, b_inv = p["b"], None, None
    if case["post"]:
        b_unit, b_inv = norm(p["b"])
        t = b_unit * p["w_post"]
    gain = case["alpha"] * p.get("scale", 1.0)
    x = p["r"] + gain * t
    unit, inv = norm(x)
    got = {"r_out": x, "h": unit * p["w"]}
    if kind == "residual_fwd":
        return got
    if case["ckpt"]:  # what is kept is the stream as it is stored
        unit = _kept64(x.to(DTYPES[case["res"]])) * inv.reshape(m, 1)
    elif case["res"] == "bf16":
        unit = x.to(torch.bfloat16).double() * inv.reshape(m, 1)
    d_x = norm_back(p["dh"] * p["w"], unit, inv) + p["dr_out"]
    d_t = gain * d_x
    got["d_r"], got["d_w"] = d_x, (p["dh"] * unit).sum(0)
    got["d_b"] = norm_back(d_t * p["w_post"], b_unit, b_inv) if case["post"] else d_t
    got["d_w_post"] = (d_t * b_unit).sum(0) if case["post"] else None
    got["d_scale"] = (case["alpha"] * d_x * t).sum(0) if case["scale"] else None
    return got
