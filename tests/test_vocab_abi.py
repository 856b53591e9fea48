"""Refusals and sizes of the losses over a vocabulary, on the CPU: every bad argument
is turned away on the host with its documented status before a launch.  Pointers
are small integers that are never followed."""
import pytest
import torch

import selective_scan_recurrence_amd as ssm
from selective_scan_recurrence_amd import ops

BIG = 1 << 44


def _status(f, *a, **kw):
    with pytest.raises(ssm.SsmError) as e:
        f(*a, **kw)
    return e.value.status


def _desc(**kw):
    return ops.vocab_desc(**{**dict(n_rows=4, width=96, n_vocab=300), **kw})


def _ce_fwd(d, **kw):
    a = dict(h=256, w=256, target=256, loss=256, lse=256, err=None, workspace=256, workspace_bytes=BIG)
    a.update(kw)
    return ssm.ssm_vocab_ce_fwd(d, *a.values(), stream=0)


def _ce_bwd(d, **kw):
    a = dict(h=256, w=256, target=256, loss=256, lse=256, d_loss=256, d_lse=None, d_h=256, d_w=256, workspace=256,
             workspace_bytes=BIG)
    a.update(kw)
    return ssm.ssm_vocab_ce_bwd(d, *a.values(), stream=0)


def _kd_fwd(d, **kw):
    a = dict(h=256, w=256, top_id=256, top_logit=256, top_lse=None, loss=256, lse=256, logq=256, err=None,
             workspace=256, workspace_bytes=BIG)
    a.update(kw)
    return ssm.ssm_vocab_kd_fwd(d, *a.values(), stream=0)


def _kd_bwd(d, **kw):
    a = dict(h=256, w=256, top_id=256, top_logit=256, top_lse=None, logq=256, lse=256, d_loss=256, d_lse=None,
             d_h=256, d_w=256, workspace=256, workspace_bytes=BIG)
    a.update(kw)
    return ssm.ssm_vocab_kd_bwd(d, *a.values(), stream=0)


CALLS = [(_ce_fwd, 0), (_ce_bwd, 0), (_kd_fwd, 3), (_kd_bwd, 3)]


@pytest.mark.parametrize("call,top", CALLS)
@pytest.mark.parametrize("field,value", [
    ("n_rows", -1), ("n_rows", (1 << 21) + 1), ("width", 0), ("width", -1), ("width", (1 << 16) + 1), ("n_vocab", 0),
    ("n_vocab", (1 << 24) + 1), ("n_top", -1), ("n_top", 1025), ("ld_h", 95), ("ld_w", 1), ("ld_h", -96),
    ("ld_w", (1 << 22) + 1), ("ld_h", 1 << 61), ("scale", float("inf")), ("scale", float("nan")),
    ("top_scale", float("nan")), ("flags", 2), ("reserved", 1),
])
def test_bad_descriptor(call, top, field, value):
    d = _desc(n_top=top)
    setattr(d, field, value)
    assert _status(call, d) == ssm.SSM_ERR_SHAPE
    assert ssm.ssm_vocab_workspace_bytes(d, 0) == 0 and ssm.ssm_vocab_workspace_bytes(d, 1) == 0


@pytest.mark.parametrize("call,top", CALLS)
def test_most_values(call, top):
    """h's values are packed eight a lane, and a launch has under 2^32 lanes."""
    assert _status(call, _desc(n_rows=(1 << 18) + 1, width=1 << 16, n_top=top)) == ssm.SSM_ERR_SHAPE
    for d in (_desc(n_rows=(1 << 18) + 1, width=1 << 16), _desc(n_rows=1 << 21, width=(1 << 13) + 1)):
        assert ssm.ssm_vocab_workspace_bytes(d, 0) == 0 and ssm.ssm_vocab_workspace_bytes(d, 1) == 0
    assert ssm.ssm_vocab_workspace_bytes(_desc(n_rows=1 << 18, width=1 << 16), 0) > 0


@pytest.mark.parametrize("call,top", CALLS)
def test_bad_dtype(call, top):
    for field in ("io_dtype", "dw_dtype"):
        d = _desc(n_top=top)
        setattr(d, field, 7)
        assert _status(call, d) == ssm.SSM_ERR_DTYPE
    assert _status(call, _desc(n_top=top, io="f32", dw="bf16")) == ssm.SSM_ERR_UNSUPPORTED


@pytest.mark.parametrize("call,top", CALLS)
def test_the_other_losses_descriptor(call, top):
    """Entries a row belong to distillation, none to cross entropy."""
    assert _status(call, _desc(n_top=0 if top else 3)) == ssm.SSM_ERR_SHAPE


@pytest.mark.parametrize("call,top,names", [
    (_ce_fwd, 0, ["h", "w", "target", "workspace"]),
    (_ce_bwd, 0, ["h", "w", "target", "loss", "lse", "d_loss", "workspace"]),
    (_kd_fwd, 3, ["h", "w", "top_id", "top_logit", "workspace"]),
    (_kd_bwd, 3, ["h", "w", "top_id", "top_logit", "logq", "lse", "d_loss", "workspace"]),
])
def test_missing_pointer(call, top, names):
    for name in names:
        assert _status(call, _desc(n_top=top), **{name: None}) == ssm.SSM_ERR_NULL, name


@pytest.mark.parametrize("call,top", CALLS)
def test_alignment(call, top):
    d = _desc(n_top=top)
    assert _status(call, d, h=257) == ssm.SSM_ERR_ALIGN
    assert _status(call, d, w=257) == ssm.SSM_ERR_ALIGN
    assert _status(call, d, workspace=272) == ssm.SSM_ERR_ALIGN
    assert _status(call, d, lse=258) == ssm.SSM_ERR_ALIGN
    assert _status(call, d, **({"top_id": 258} if top else {"target": 258})) == ssm.SSM_ERR_ALIGN
    assert _status(call, _desc(n_top=top, io="f32"), h=258) == ssm.SSM_ERR_ALIGN
    if call in (_ce_bwd, _kd_bwd):
        assert _status(call, d, d_h=257) == ssm.SSM_ERR_ALIGN
        assert _status(call, d, d_w=258) == ssm.SSM_ERR_ALIGN  # f32


@pytest.mark.parametrize("call,top", CALLS)
@pytest.mark.parametrize("n", [4, 500])
def test_short_workspace(call, top, n):
    d = _desc(n_top=top, n_rows=n)
    need = ssm.ssm_vocab_workspace_bytes(d, int(call in (_ce_bwd, _kd_bwd)))
    assert need > 0 and need % 256 == 0
    assert _status(call, d, workspace_bytes=need - 1) == ssm.SSM_ERR_WORKSPACE


def test_a_backwards_workspace_serves_the_forward():
    for kw in (dict(), dict(n_rows=1), dict(n_rows=70, width=65536, n_vocab=5000, io="f32"), dict(n_rows=16384, n_vocab=1 << 20)):
        d = _desc(**kw)
        assert ssm.ssm_vocab_workspace_bytes(d, 1) >= ssm.ssm_vocab_workspace_bytes(d, 0)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_workspace_stays_small(io):
    """The vocabulary's pieces bound it: about 1.25 GiB and the rows' own tensors, where
    the logits of 16384 rows would take 64 GiB in f32."""
    d = _desc(n_rows=16384, width=2560, n_vocab=1 << 20, io=io)
    assert ssm.ssm_vocab_workspace_bytes(d, 1) < 3 << 30
    assert ssm.ssm_vocab_workspace_bytes(d, 0) < 3 << 30


def test_nothing_to_do():
    """No rows and no gradient asked for: nothing is launched."""
    _ce_fwd(_desc(n_rows=0), h=None, target=None)
    _kd_fwd(_desc(n_rows=0, n_top=2), h=None, top_id=None, top_logit=None)
    _ce_bwd(_desc(), d_h=None, d_w=None)
    _kd_bwd(_desc(n_top=2), d_h=None, d_w=None)


@pytest.mark.parametrize("call,top", CALLS)
@pytest.mark.parametrize("scale", [2.4e38, -3.0e38])
def test_scale_times_log2_e_is_finite(call, top, scale):
    """The kernels' logits are times log2 e; a teacher's scale is not."""
    assert _status(call, _desc(n_top=top, scale=scale)) == ssm.SSM_ERR_SHAPE
    assert ssm.ssm_vocab_workspace_bytes(_desc(n_top=top, scale=scale), 1) == 0
    assert ssm.ssm_vocab_workspace_bytes(_desc(n_top=top, scale=1.7e38, top_scale=scale), 1) > 0


def test_strides_default_to_dense():
    d = ssm.SsmVocabDesc(4, 96, 300, 0, 0, 0, ssm.SSM_BF16, ssm.SSM_F32, 1.0, 1.0, 0, 0)
    assert ssm.ssm_vocab_workspace_bytes(d, 1) == ssm.ssm_vocab_workspace_bytes(_desc(), 1)


# ---- what the C ABI cannot see ----------------------------------------------------


def _on(index, *shape, dtype=torch.float32):
    """A tensor that says it is on GPU index; it has no memory."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        return torch.empty(*shape, dtype=dtype, device=f"cuda:{index}")


class _Stream:
    """A stream of GPU 1."""
    device_index, cuda_stream = 1, 256


F, I, IO, U8 = torch.float32, torch.int32, torch.bfloat16, torch.uint8


def _arguments(name):
    """A complete call of ops.<name>: its descriptor, and its tensors by name with their
    shapes and types."""
    row, top, h, w = ((4,), F), ((4, 3), F), ((4, 96), IO), ((300, 96), IO)
    ws = ((1 << 24,), U8)
    lead = dict(h=h, w=w)
    ids = dict(target=((4,), I)) if "ce" in name else dict(top_id=((4, 3), I), top_logit=top)
    if name.endswith("fwd"):
        rest = dict(loss=row, lse=row, err=((1,), I), ws=ws)
        rest.update({} if "ce" in name else dict(logq=top, top_lse=row))
    else:
        rest = dict(loss=row) if "ce" in name else dict(logq=top, top_lse=row)
        rest.update(lse=row, d_loss=row, d_lse=row, d_h=h, d_w=((300, 96), F), ws=ws)
    return _desc(n_top=0 if "ce" in name else 3), {**lead, **ids, **rest}


NAMES = ["vocab_ce_fwd", "vocab_ce_bwd", "vocab_kd_fwd", "vocab_kd_bwd"]


def _call_with(name, home, odd, tensor, **kw):
    desc, tensors = _arguments(name)
    args = {k: tensor if k == odd else _on(home, *shape, dtype=dtype) for k, (shape, dtype) in tensors.items()}
    with pytest.raises(ssm.SsmError, match=rf": {odd} is ") as e:
        getattr(ops, name)(desc, **args, **kw)
    return e.value.status


@pytest.mark.parametrize("where", ["cpu", "other", "stream"])
@pytest.mark.parametrize("name", NAMES)
def test_tensors_are_on_the_device_of_the_launch(monkeypatch, name, where):
    monkeypatch.setattr(ops, "_current_device", lambda: 0, raising=False)
    home = 1 if where == "stream" else 0
    for odd, (shape, dtype) in _arguments(name)[1].items():
        t = torch.empty(*shape, dtype=dtype) if where == "cpu" else _on(1 - home, *shape, dtype=dtype)
        kw = dict(stream=_Stream()) if where == "stream" else {}
        assert _call_with(name, home, odd, t, **kw) == ssm.SSM_ERR_UNSUPPORTED, odd


@pytest.mark.parametrize("name", NAMES)
def test_types_and_layouts_are_checked(monkeypatch, name):
    monkeypatch.setattr(ops, "_current_device", lambda: 0, raising=False)
    for odd, (shape, dtype) in _arguments(name)[1].items():
        if odd == "ws":
            continue
        other = torch.int64 if dtype is I else torch.float64
        assert _call_with(name, 0, odd, _on(0, *shape, dtype=other)) == ssm.SSM_ERR_DTYPE, odd
        short = (shape[0] - 1,) + shape[1:]
        assert _call_with(name, 0, odd, _on(0, *short, dtype=dtype)) == ssm.SSM_ERR_SHAPE, odd
        if len(shape) == 2:  # transposed; rows that share memory; a stride that is not the descriptor's
            assert _call_with(name, 0, odd, _on(0, *shape[::-1], dtype=dtype).t()) == ssm.SSM_ERR_SHAPE, odd
            assert _call_with(name, 0, odd, _on(0, 1, shape[1], dtype=dtype).expand(*shape)) == ssm.SSM_ERR_SHAPE, odd
            wide = _on(0, shape[0], shape[1] + 8, dtype=dtype)[:, :shape[1]]
            assert _call_with(name, 0, odd, wide) == ssm.SSM_ERR_SHAPE, odd


def test_accumulate_needs_a_gradient(monkeypatch):
    monkeypatch.setattr(ops, "_current_device", lambda: 0, raising=False)
    _, tensors = _arguments("vocab_ce_bwd")
    args = {k: _on(0, *shape, dtype=dtype) for k, (shape, dtype) in tensors.items() if k != "d_w"}
    assert _status(ops.vocab_ce_bwd, _desc(accumulate=True), **args) == ssm.SSM_ERR_NULL
