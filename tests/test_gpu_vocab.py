"""The losses over a vocabulary against the 64-bit reference: every shape of
tile, ends of rows, vocabulary and width, types, strides and rows left out."""
import pytest
import torch

import vocab_ref as R
from block_ref import padding_untouched, strided
from selective_scan_recurrence_amd import ops

pytestmark = pytest.mark.gpu

# rows, width, vocabulary
SIZES = [(1, 64, 1), (1, 1, 5), (1, 64, 300), (3, 40, 77), (16, 128, 1000), (17, 130, 513), (33, 2560, 1030),
         (64, 64, 256), (65, 72, 4097), (130, 192, 700), (257, 100, 515), (300, 515, 640), (520, 64, 130),
         (70, 320, 9001), (20, 72, 26001), (40, 100, 13001), (64, 33, 30001), (32, 200, 12801), (128, 128, 1000), (9, 65, 26000),
         (100, 1100, 7000), (3, 1500, 26003)]


def run(t, io, *, dw="f32", scale=1.0, top_scale=1.0, pad_h=0, pad_w=0, d_lse=None, top_lse=None, d_w0=None,
        ws=None, stream=None, err=None):
    """A forward and a backward; the results by name."""
    n, d = t["h"].shape
    v = t["w"].shape[0]
    h, w = strided(t["h"], pad_h, R.DTYPES[io]), strided(t["w"], pad_w, R.DTYPES[io])
    top = t["top_id"].shape[1] if "top_id" in t else 0
    desc = ops.vocab_desc(n_rows=n, width=d, n_vocab=v, n_top=top, io=io, dw=dw, scale=scale, top_scale=top_scale,
                          ld_h=d + pad_h, ld_w=d + pad_w, accumulate=d_w0 is not None)
    kw = dict(ws=ws, stream=stream)
    bk = dict(kw, d_h=strided(torch.zeros(n, d), pad_h, R.DTYPES[io]),
              d_w=strided(torch.zeros(v, d) if d_w0 is None else d_w0, pad_w, R.DTYPES[dw]),
              d_lse=None if d_lse is None else d_lse.cuda())
    if top:
        ids, logit = t["top_id"].cuda(), t["top_logit"].cuda()
        lse = None if top_lse is None else top_lse.cuda()
        f = ops.vocab_kd_fwd(desc, h, w, ids, logit, top_lse=lse, err=err, **kw)
        g = ops.vocab_kd_bwd(desc, h, w, ids, logit, f.logq, f.lse, t["d_loss"].cuda(), top_lse=lse, **bk)
    else:
        target = t["target"].cuda()
        f = ops.vocab_ce_fwd(desc, h, w, target, err=err, **kw)
        g = ops.vocab_ce_bwd(desc, h, w, target, f.loss, f.lse, t["d_loss"].cuda(), **bk)
    torch.cuda.synchronize()
    assert padding_untouched(g.d_h) and padding_untouched(g.d_w)
    return {"loss": f.loss, "lse": f.lse, "logq": f.logq, "d_h": g.d_h, "d_w": g.d_w}


def compare(t, io, got, *, dw="f32", scale=1.0, top_scale=1.0, d_lse=None, top_lse=None, d_w0=None):
    ref = R.Reference(t["h"], t["w"], io, target=t.get("target"), top_id=t.get("top_id"),
                      top_logit=t.get("top_logit"), top_lse=top_lse, scale=scale, top_scale=top_scale)
    want = {**ref.forward(), **ref.backward(t["d_loss"], d_lse, dw, d_w0)}
    if got["logq"] is None:
        del want["logq"]
    for name, (value, err) in want.items():
        R.check(name, got[name], value, err)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,d,v", SIZES)
def test_cross_entropy(n, d, v, io):
    t = R.problem(n + d + v, n, d, v, io, out=0.3 if n > 4 else 0.0)
    compare(t, io, run(t, io))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("top", [1, 2, 7, 33, 100])
@pytest.mark.parametrize("n,d,v", [(1, 64, 300), (17, 130, 513), (130, 192, 700), (65, 72, 4097)])
def test_distillation(n, d, v, top, io):
    t = R.problem(n + d + v + top, n, d, v, io, top=top, out=0.2 if n > 4 else 0.0)
    compare(t, io, run(t, io, scale=0.5, top_scale=0.7), scale=0.5, top_scale=0.7)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_teacher_as_it_stands(io):
    t = R.problem(5, 70, 96, 600, io, top=9, out=0.1)
    top_lse = torch.logsumexp(t["top_logit"], 1) + 0.25
    compare(t, io, run(t, io, top_lse=top_lse), top_lse=top_lse)


@pytest.mark.parametrize("pad_h,pad_w", [(0, 1), (1, 0), (8, 64), (3, 8)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_strides(io, pad_h, pad_w):
    """Slices of wider tensors; what lies behind their rows stays as it was."""
    t = R.problem(11, 70, 128, 300, io, out=0.2)
    compare(t, io, run(t, io, pad_h=pad_h, pad_w=pad_w))


@pytest.mark.parametrize("top", [0, 5])
def test_bf16_weight_gradient(top):
    t = R.problem(12, 70, 129, 300, "bf16", top=top, out=0.2)
    compare(t, "bf16", run(t, "bf16", dw="bf16"), dw="bf16")


@pytest.mark.parametrize("dw,io", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
def test_accumulates(dw, io):
    t = R.problem(13, 70, 130, 300, io)
    d_w0 = (0.1 * torch.randn(300, 130, generator=torch.Generator().manual_seed(1))).to(R.DTYPES[dw])
    compare(t, io, run(t, io, dw=dw, d_w0=d_w0), dw=dw, d_w0=d_w0)


@pytest.mark.parametrize("top", [0, 4])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_gradient_of_lse(io, top):
    t = R.problem(14, 66, 96, 300, io, top=top, out=0.2)
    d_lse = 0.05 * torch.randn(66, generator=torch.Generator().manual_seed(2))
    compare(t, io, run(t, io, scale=1.5, d_lse=d_lse), scale=1.5, d_lse=d_lse)


@pytest.mark.parametrize("top", [0, 6])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 40, 300])
def test_no_row_counts(n, top, io):
    t = R.problem(15, n, 64, 300, io, top=top, out=2.0)
    t["h"][:], t["d_loss"][:] = float("nan"), float("nan")
    compare(t, io, run(t, io))


@pytest.mark.parametrize("top", [0, 6])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n", [9, 300])
def test_rows_left_out_may_hold_anything(n, top, io):
    t = R.problem(16, n, 96, 300, io, top=top, out=0.5)
    out = (t["target"] < 0) if not top else (t["top_id"] < 0).all(1)
    assert bool(out.any()) and not bool(out.all())
    t["h"][out] = torch.tensor([float("nan"), float("inf"), -float("inf")]).repeat(32).to(t["h"].dtype)
    t["d_loss"][out] = float("nan")
    d_lse = torch.where(out, float("inf"), 0.01)
    if top:
        t["top_logit"][t["top_id"] < 0] = float("nan")
    compare(t, io, run(t, io, d_lse=d_lse), d_lse=d_lse)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_no_rows(io):
    """n_rows = 0: no loss, and a weight gradient of zeros."""
    w = torch.randn(300, 64).to(R.DTYPES[io]).cuda()
    empty = torch.zeros(0, 64, dtype=w.dtype, device="cuda")
    none, none_i = torch.zeros(0, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    desc = ops.vocab_desc(n_rows=0, width=64, n_vocab=300, io=io)
    f = ops.vocab_ce_fwd(desc, empty, w, none_i)
    g = ops.vocab_ce_bwd(desc, empty, w, none_i, f.loss, f.lse, none)
    assert f.loss.shape == (0,) and g.d_h.shape == (0, 64) and bool((g.d_w == 0).all())


@pytest.mark.parametrize("top", [0, 3])
@pytest.mark.parametrize("n", [5, 140])
def test_ids_past_the_vocabulary(n, top):
    t = R.problem(17, n, 64, 300, "bf16", top=top)
    if top:
        t["top_id"][2, 1], t["top_id"][4, 2] = 300, 2 ** 31 - 1
    else:
        t["target"][2], t["target"][4] = 300, 2 ** 31 - 1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    compare(t, "bf16", run(t, "bf16", err=err))
    import selective_scan_recurrence_amd as ssm
    assert int(err.item()) == ssm.SSM_DEVERR_TARGET


def test_same_id_twice():
    t = R.problem(18, 40, 64, 300, "f32", top=6)
    t["top_id"][:, 3] = t["top_id"][:, 1]
    t["top_id"][:20, 5] = t["top_id"][:20, 1]
    compare(t, "f32", run(t, "f32"))


def test_entries_without_mass():
    """A logit of -inf is no entry, wherever its id points; a row of them is left out."""
    t = R.problem(19, 40, 64, 300, "f32", top=4)
    t["top_logit"][::3, 1] = -float("inf")
    t["top_id"][::3, 1] = 10 ** 9
    t["top_logit"][5] = -float("inf")
    compare(t, "f32", run(t, "f32"))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n", [3, 200])
def test_logits_far_from_zero(n, io):
    """All logits of a row far below or above zero, a vocabulary that ends inside a
    tile: nothing but the row's own logits enters its softmax."""
    t = R.problem(20, n, 64, 333, io)
    t["w"] = t["w"].abs()
    t["h"] = (t["h"].float().abs() * torch.where(torch.arange(n) % 2 == 0, -40.0, 40.0)[:, None]).to(R.DTYPES[io])
    compare(t, io, run(t, io))


def test_infinite_and_nan_rows_stay_alone():
    """A NaN or infinite row of h makes its own loss and d_h NaN, not its neighbours'."""
    t = R.problem(21, 70, 64, 300, "bf16")
    t["h"][7, 3], t["h"][33, 0] = float("nan"), float("inf")
    got = run(t, "bf16")
    rest = torch.ones(70, dtype=torch.bool)
    rest[[7, 33]] = False
    assert not bool(torch.isfinite(got["loss"].cpu()[~rest]).any())
    assert bool(got["d_h"].float().cpu()[~rest].isnan().any(1).all())
    fine = {k: v[rest] if v.shape[0] == 70 else v for k, v in t.items()}
    alone = run(fine, "bf16")
    for name in ("loss", "lse", "d_h"):
        assert torch.equal(got[name].cpu()[rest], alone[name].cpu()), name


def test_teacher_that_agrees():
    """The loss of a teacher that equals the student is zero within rounding."""
    t = R.problem(22, 33, 64, 40, "f32", top=40)
    s = t["h"].double() @ t["w"].double().t()
    t["top_id"] = torch.arange(40).repeat(33, 1).int()
    t["top_logit"] = s.float()
    compare(t, "f32", run(t, "f32"))


def test_vocabulary_in_pieces():
    """A workspace of a gigabyte holds 2560 entries of 65536 columns in f32, and fewer
    with the gradient's tensors: the vocabulary goes through in pieces."""
    t = R.problem(23, 3, 65536, 3001, "f32")
    compare(t, "f32", run(t, "f32"))


def test_repeats_bitwise():
    t = R.problem(24, 300, 200, 2000, "bf16", top=8, out=0.2)
    a, b = run(t, "bf16"), run(t, "bf16")
    for name in a:
        assert torch.equal(a[name], b[name]), name


def test_only_one_gradient():
    t = R.problem(25, 70, 128, 300, "bf16")
    both = run(t, "bf16")
    desc = ops.vocab_desc(n_rows=70, width=128, n_vocab=300)
    h, w, target, d = (t[k].cuda() for k in ("h", "w", "target", "d_loss"))
    f = ops.vocab_ce_fwd(desc, h, w, target)
    gh = ops.vocab_ce_bwd(desc, h, w, target, f.loss, f.lse, d, want_w=False)
    gw = ops.vocab_ce_bwd(desc, h, w, target, f.loss, f.lse, d, want_h=False)
    assert gh.d_w is None and gw.d_h is None
    assert torch.equal(gh.d_h, both["d_h"]) and torch.equal(gw.d_w, both["d_w"])
