"""The losses over a vocabulary where it is long for its rows: many parts of d_h's sum,
and several pieces of the vocabulary.  The reference runs on the GPU, in 64 bits."""
import pytest
import torch

import selective_scan_recurrence_amd as ssm
import vocab_ref as R
from selective_scan_recurrence_amd import ops
from test_gpu_vocab import compare, run

pytestmark = pytest.mark.gpu


def _on_gpu(*a, **kw):
    return {k: v.cuda() for k, v in R.problem(*a, **kw).items()}


@pytest.mark.parametrize("n,d,v,io,out", [(100, 64, 66000, "bf16", 0.0), (100, 64, 131072, "bf16", 0.5),
                                          (65, 64, 1 << 20, "bf16", 0.0), (128, 128, 131072, "f32", 0.1)])
@pytest.mark.parametrize("both", [True, False])
def test_parts_of_a_long_vocabulary(n, d, v, io, out, both):
    t = _on_gpu(n + v, n, d, v, io, out=out)
    if both:
        return compare(t, io, run(t, io))
    desc = ops.vocab_desc(n_rows=n, width=d, n_vocab=v, io=io)
    f = ops.vocab_ce_fwd(desc, t["h"], t["w"], t["target"])
    g = ops.vocab_ce_bwd(desc, t["h"], t["w"], t["target"], f.loss, f.lse, t["d_loss"], want_w=False)
    want = R.Reference(t["h"], t["w"], io, target=t["target"]).backward(t["d_loss"])
    R.check("d_h", g.d_h, *want["d_h"])


# ---- pieces of the vocabulary -------------------------------------------------------


def _in_pieces(backward, v, less, **kw):
    """Whether v goes through in several pieces: where the piece's tensors are most of the
    workspace, it then takes less of it than the shorter vocabulary `less`."""
    def size(n):
        return ssm.ssm_vocab_workspace_bytes(ops.vocab_desc(n_vocab=n, **kw), backward)
    assert less < v
    return size(v) < size(less)


def _check(what, got, want, err):
    """R.check where the tensors are."""
    got = got.double().reshape(want.shape)
    assert torch.equal(got.isnan(), want.isnan()), what
    off = torch.where(want.isnan(), 0.0, (got - want).abs() - err.expand_as(want))
    assert bool((off <= 0).all()), f"{what}: {int((~(off <= 0)).sum())} of {off.numel()} outside, by {float(off.max())}"


def _check_all(t, io, got, **kw):
    ref = R.Reference(t["h"], t["w"], io, target=t.get("target"), top_id=t.get("top_id"),
                      top_logit=t.get("top_logit"))
    for name, (value, err) in {**ref.forward(), **ref.backward(t["d_loss"], **kw)}.items():
        if got[name] is not None:
            _check(name, got[name], value, err)


WIDE = dict(n=70, d=65536, v=3400)  # f32: W's terms take 393 KB an entry


def _wide(top):
    """The forward goes through the vocabulary in two pieces, the backward in three."""
    kw = dict(n_rows=WIDE["n"], width=WIDE["d"], n_top=top, io="f32")
    return _in_pieces(0, WIDE["v"], 3328, **kw) and _in_pieces(1, WIDE["v"], 1536, **kw)


@pytest.mark.parametrize("top", [0, 5])
def test_wide_rows(top):
    n, d, v = WIDE.values()
    assert _wide(top)
    gen = torch.Generator(device="cuda").manual_seed(50 + top)
    w = torch.randn(v, d, generator=gen, device="cuda") * (2.5 / d ** 0.5)
    small = R.problem(51, n, 1, v, "f32", top=top, out=0.2)
    t = {k: x.cuda() for k, x in small.items() if k not in ("h", "w")}
    first = (t["top_id"][:, 0] if top else t["target"]).long().clamp(min=0)
    t["w"], t["h"] = w, torch.randn(n, d, generator=gen, device="cuda") + w[first]
    _check_all(t, "f32", run(t, "f32"))
    torch.cuda.empty_cache()


@pytest.mark.parametrize("top", [0, 5])
def test_wide_rows_of_few_values(top):
    """64 of the columns hold values and the rest zeros, whose products and sums are exact:
    within the bounds of a width of 64, which a piece left out or counted twice passes."""
    n, d, v = WIDE.values()
    assert _wide(top)
    t = _on_gpu(52 + top, n, 64, v, "f32", top=top, out=0.2)
    columns = torch.randperm(d, generator=torch.Generator().manual_seed(top))[:64].cuda()
    wide = dict(t, h=torch.zeros(n, d, device="cuda"), w=torch.zeros(v, d, device="cuda"))
    wide["h"][:, columns], wide["w"][:, columns] = t["h"], t["w"]
    got = run(wide, "f32")
    for name in ("d_h", "d_w"):
        mine = got[name][:, columns]
        got[name][:, columns] = 0.0
        assert bool((got[name] == 0).all()), name
        got[name] = mine
    _check_all(t, "f32", got)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("top", [0, 5])
@pytest.mark.parametrize("dw,add", [("f32", False), ("bf16", True)])
def test_many_rows_in_bf16(top, dw, add):
    """4000 rows: g takes 17 KB an entry, and the backward goes through 90000 of the
    vocabulary in two pieces, d_h added up over them."""
    n, d, v = 4000, 72, 90000
    assert _in_pieces(1, v, 74000, n_rows=n, width=d, n_top=top, dw=dw)
    t = _on_gpu(52 + top, n, d, v, "bf16", top=top, out=0.2)
    kw = {}
    if add:
        kw["d_w0"] = 1e-4 * torch.randn(v, d, generator=torch.Generator().manual_seed(6)).to(R.DTYPES[dw])
    got = run(t, "bf16", dw=dw, **kw)
    if add:
        kw["d_w0"] = kw["d_w0"].cuda()
    _check_all(t, "bf16", got, dw=dw, **kw)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("io,v,less", [("bf16", 2700000, 2620000), ("f32", 1800001, 1747000)])
@pytest.mark.parametrize("top", [0, 5])
@pytest.mark.parametrize("n,add", [(1, False), (5, True), (40, False)])
def test_few_rows(n, io, v, less, top, add):
    """Up to 64 rows: both of g's orders take 512 bytes an entry, 768 in f32."""
    d = 8
    assert _in_pieces(1, v, less, n_rows=n, width=d, n_top=top, io=io)
    t = _on_gpu(60 + n + top, n, d, v, io, top=top, out=0.2 if n > 1 else 0.0)
    kw = {}
    if add:
        kw["d_w0"] = 1e-4 * torch.randn(v, d, generator=torch.Generator().manual_seed(7))
    got = run(t, io, **kw)
    if add:
        kw["d_w0"] = kw["d_w0"].cuda()
    _check_all(t, io, got, **kw)
    torch.cuda.empty_cache()
