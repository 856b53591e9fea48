"""Torch-level convenience over the C ABI: builds descriptors, allocates the
packed outputs and workspaces as torch device tensors, and splits packed
results into views.  Every computation runs in libssm.so's HIP kernels;
torch only provides memory and the stream.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from . import _binding as B

IO_DTYPES = {"f32": B.SSM_F32, "bf16": B.SSM_BF16}
TORCH_IO = {B.SSM_F32: torch.float32, B.SSM_BF16: torch.bfloat16}


def make_desc(*, n_seqs, n_tokens, n_head, d_state, head_dim=1, n_group=1, n_state_rows=None,
              a_per_state=True, d_conv=0, chunk=0, io="f32", has_D=True,
              dt_softplus=False) -> B.SsmScanDesc:
    flags = (B.SSM_HAS_D if has_D else 0) | (B.SSM_DT_SOFTPLUS if dt_softplus else 0)
    return B.SsmScanDesc(int(n_seqs), int(n_tokens), int(n_head), int(head_dim), int(d_state),
                         int(n_group), int(n_seqs if n_state_rows is None else n_state_rows),
                         int(bool(a_per_state)), int(d_conv), int(chunk),
                         IO_DTYPES[io] if isinstance(io, str) else int(io), int(flags), 0)


def workspace(desc: B.SsmScanDesc, backward: bool, device="cuda") -> torch.Tensor:
    """A zeroed workspace (its first word is the sticky device-error word)."""
    n = B.ssm_scan_workspace_bytes(desc, int(backward))
    if n == 0:
        raise B.SsmError(B.SSM_ERR_SHAPE, "ssm_scan_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


@dataclass
class FwdResult:
    out: torch.Tensor            # packed bytes: y | state
    y: torch.Tensor              # view [n_seqs][n_tokens][n_head][head_dim], io dtype
    state: torch.Tensor          # view [n_seqs][n_head][head_dim][d_state], f32
    conv_state: Optional[torch.Tensor]


def split_out(desc: B.SsmScanDesc, out: torch.Tensor):
    io = TORCH_IO[desc.io_dtype]
    off = B.ssm_scan_state_offset_bytes(desc)
    n_y = desc.n_seqs * desc.n_tokens * desc.n_head * desc.head_dim
    y = out[:off].view(io)[:n_y].view(desc.n_seqs, desc.n_tokens, desc.n_head, desc.head_dim)
    st = out[off:].view(torch.float32).view(desc.n_seqs, desc.n_head, desc.head_dim, desc.d_state)
    return y, st


def scan_fwd(desc, s, x, dt, A, Bm, Cm, D, ids, conv_w=None, conv_state=None,
             want_conv_state=False, ws=None, out=None, stream=None) -> FwdResult:
    if out is None:
        out = torch.empty(B.ssm_scan_out_bytes(desc), dtype=torch.uint8, device=x.device)
    cso = None
    if want_conv_state and desc.d_conv > 1:
        cso = torch.empty(desc.n_seqs, desc.n_head, desc.d_conv - 1, dtype=torch.float32,
                          device=x.device)
    if ws is None:
        ws = workspace(desc, False, x.device)
    B.selective_scan_fwd(desc, s, x, dt, A, Bm, Cm, D, ids, conv_w, conv_state, out, cso, ws,
                         ws.numel(), stream)
    y, st = split_out(desc, out)
    return FwdResult(out, y, st, cso)


def scan_fwd_ext(desc, s, x, dt, A, Bm, Cm, D, ids, *, dt_bias=None, z=None, cu_seqlens=None,
                 total_tokens=0, conv_w=None, conv_state=None, want_conv_state=False, ws=None,
                 out=None, stream=None) -> FwdResult:
    """selective_scan_fwd_ext.  With cu_seqlens (int32 device [n_seqs+1]) the
    token axis is packed: y is returned as [total_tokens][n_head][head_dim]."""
    ext = B.make_ext(dt_bias, z, cu_seqlens, total_tokens if cu_seqlens is not None else 0)
    total, off = B.ssm_scan_ext_out_bytes(desc, ext)
    if total == 0:
        raise B.SsmError(B.SSM_ERR_SHAPE, "ssm_scan_ext_out_bytes")
    if out is None:
        out = torch.empty(total, dtype=torch.uint8, device=x.device)
    cso = None
    if want_conv_state and desc.d_conv > 1:
        cso = torch.empty(desc.n_seqs, desc.n_head, desc.d_conv - 1, dtype=torch.float32,
                          device=x.device)
    if ws is None:
        ws = workspace(desc, False, x.device)
    B.selective_scan_fwd_ext(desc, ext, s, x, dt, A, Bm, Cm, D, ids, conv_w, conv_state, out, cso,
                             ws, ws.numel(), stream)
    io = TORCH_IO[desc.io_dtype]
    H, P = desc.n_head, desc.head_dim
    n_tok = total_tokens if cu_seqlens is not None else desc.n_seqs * desc.n_tokens
    y = out[:off].view(io)[:n_tok * H * P].view(n_tok, H, P)
    if cu_seqlens is None:
        y = y.view(desc.n_seqs, desc.n_tokens, H, P)
    st = out[off:].view(torch.float32).view(desc.n_seqs, H, P, desc.d_state)
    return FwdResult(out, y, st, cso)


def split_dgrad(desc: B.SsmScanDesc, dgrad: torch.Tensor) -> dict:
    """Views of the packed gradient: d_s, d_x, d_dt, d_A, d_B, d_C, d_D (with
    D), then d_conv_w and d_conv_state (with the fused conv)."""
    total, offs = B.ssm_scan_dgrad_layout(desc)
    S, L, H, P, N, G, R, K = (desc.n_seqs, desc.n_tokens, desc.n_head, desc.head_dim,
                              desc.d_state, desc.n_group, desc.n_state_rows, desc.d_conv)
    shapes = {"d_s": (R, H, P, N), "d_x": (S, L, H, P), "d_dt": (S, L, H),
              "d_A": (H, N) if desc.a_per_state else (H,), "d_B": (S, L, G, N),
              "d_C": (S, L, G, N)}
    if desc.flags & B.SSM_HAS_D:
        shapes["d_D"] = (H,)
    if K > 0:
        shapes["d_conv_w"] = (H, K)
        shapes["d_conv_state"] = (R, H, K - 1)
    res = {}
    off = 0
    for name, shape in shapes.items():
        n = 1
        for v in shape:
            n *= v
        res[name] = dgrad[off:off + 4 * n].view(torch.float32).view(*shape)
        off += 4 * n
    assert off == total, (off, total)
    return res


def scan_bwd(desc, s, x, dt, A, Bm, Cm, D, ids, dout, ws=None, dgrad=None, stream=None,
             conv_w=None, conv_state=None):
    """Returns (packed dgrad bytes, dict of views).  With the fused conv
    (desc.d_conv > 0) conv_w is required and conv_state optional (zeros);
    the call is selective_scan_bwd_conv and d_x is the gradient of the
    pre-conv input."""
    total, _ = B.ssm_scan_dgrad_layout(desc)
    if dgrad is None:
        dgrad = torch.empty(total, dtype=torch.uint8, device=x.device)
    if ws is None:
        ws = workspace(desc, True, x.device)
    if desc.d_conv > 0 or conv_w is not None:
        B.selective_scan_bwd_conv(desc, s, x, dt, A, Bm, Cm, D, ids, conv_w, conv_state, dout, dgrad,
                                  ws, ws.numel(), stream)
    else:
        B.selective_scan_bwd(desc, s, x, dt, A, Bm, Cm, D, ids, dout, dgrad, ws, ws.numel(), stream)
    return dgrad, split_dgrad(desc, dgrad)


def conv_fwd(sx: torch.Tensor, w: torch.Tensor, apply_silu=False, out=None, stream=None):
    """ggml ssm_conv: sx [n_s][d_inner][d_conv-1+n_t], w [d_inner][d_conv] ->
    out [n_s][n_t][d_inner] (sx's dtype)."""
    n_s, d_inner, length = sx.shape
    d_conv = w.shape[1]
    n_t = length - (d_conv - 1)
    io = B.SSM_BF16 if sx.dtype == torch.bfloat16 else B.SSM_F32
    if out is None:
        out = torch.empty(n_s, n_t, d_inner, dtype=sx.dtype, device=sx.device)
    B.ssm_conv_fwd(sx, w, out, n_s, n_t, d_inner, d_conv, io, int(bool(apply_silu)), stream)
    return out


def conv_bwd_workspace(n_s, n_t, d_inner, d_conv, device="cuda") -> torch.Tensor:
    n = B.ssm_conv_bwd_workspace_bytes(n_s, n_t, d_inner, d_conv)
    return torch.empty(max(n, 4), dtype=torch.uint8, device=device)


def conv_bwd(sx: torch.Tensor, w: torch.Tensor, dout: torch.Tensor, apply_silu=False, ws=None,
             dgrad=None, stream=None):
    """Backward of ``conv_fwd``: dout [n_s][n_t][d_inner] (f32) ->
    (d_sx [n_s][d_inner][d_conv-1+n_t], d_w [d_inner][d_conv]), both f32
    views of one packed buffer (d_sx then d_w)."""
    n_s, d_inner, length = sx.shape
    d_conv = w.shape[1]
    n_t = length - (d_conv - 1)
    io = B.SSM_BF16 if sx.dtype == torch.bfloat16 else B.SSM_F32
    if ws is None:
        ws = conv_bwd_workspace(n_s, n_t, d_inner, d_conv, sx.device)
    if dgrad is None:
        dgrad = torch.empty(n_s * d_inner * length + d_inner * d_conv, dtype=torch.float32,
                            device=sx.device)
    B.ssm_conv_bwd(sx, w, dout, dgrad, n_s, n_t, d_inner, d_conv, io, int(bool(apply_silu)), ws,
                   ws.numel(), stream)
    n_sx = n_s * d_inner * length
    return dgrad[:n_sx].view(n_s, d_inner, length), dgrad[n_sx:n_sx + d_inner * d_conv].view(d_inner, d_conv)


def state_update(desc, s, x, dt, A, Bm, Cm, D, ids, *, dt_bias=None, z=None, conv_w=None,
                 conv_state=None, y=None, err=None, stream=None) -> torch.Tensor:
    """One decode token of every sequence (selective_state_update): s and
    conv_state are updated in place; returns y [n_seqs][n_head][head_dim]."""
    if y is None:
        y = torch.empty(desc.n_seqs, desc.n_head, desc.head_dim, dtype=TORCH_IO[desc.io_dtype],
                        device=s.device)
    B.selective_state_update(desc, s, x, dt, dt_bias, A, Bm, Cm, D, z, ids, conv_w, conv_state, y,
                             err, stream)
    return y


# ---- around the scan in a block: norms, 8-bit checkpoints, weight gradient ----
#
# These take [n_rows][width] tensors whose last axis is contiguous; the row
# stride may be larger (a slice of the projection's output).  What the C ABI
# cannot see of a tensor -- its shape, strides, type and device -- is checked
# here, with the ABI's status codes.  A call launches on its stream's device,
# without a stream (or with one given by its address) on the current one, and
# every tensor has to be there.


def _refuse(status, where, name, t):
    raise B.SsmError(status, f"{where}: {name} is {tuple(t.shape)} {t.dtype} on {t.device}, "
                             f"strides {t.stride()}")


_current_device = None


def _find_current_device():
    """A function that gives the current GPU's index, -2 (which no tensor has)
    where there is none.  torch's own raw getter takes 0.1 us."""
    if not torch.cuda.is_available():
        return lambda: -2
    return getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _device_of(stream):
    """Index of the GPU that a call on this stream launches on."""
    if stream is not None:
        index = getattr(stream, "device_index", None)
        if index is not None:
            return index
    global _current_device
    if _current_device is None:
        _current_device = _find_current_device()
    return _current_device()


def _matrix(where, name, t, rows, width, ld, dtype, dev=None):
    """t is None or [rows][width] in dtype with row stride ld (0: width, as the
    library takes it) on GPU dev.  Rows that share or overlap have no such
    stride."""
    if t is None:
        return
    if t.dtype is not dtype:
        _refuse(B.SSM_ERR_DTYPE, where, name, t)
    ld = ld or width
    if t.shape != (rows, width):
        _refuse(B.SSM_ERR_SHAPE, where, name, t)
    if t.stride() != (ld, 1) or ld < width:
        # neither one row's stride nor one column's matters
        if (rows > 1 and (t.stride(0) != ld or ld < width)) or \
                (width > 1 and rows > 0 and t.stride(1) != 1):
            _refuse(B.SSM_ERR_SHAPE, where, name, t)
    if t.get_device() != (_device_of(None) if dev is None else dev):
        _refuse(B.SSM_ERR_UNSUPPORTED, where, name, t)


def _dense(where, name, t, numel, dtype, dev=None):
    """t is None or a contiguous tensor of at least numel elements on GPU dev."""
    if t is None:
        return
    if t.dtype is not dtype:
        _refuse(B.SSM_ERR_DTYPE, where, name, t)
    if t.numel() < numel or not t.is_contiguous():
        _refuse(B.SSM_ERR_SHAPE, where, name, t)
    if t.get_device() != (_device_of(None) if dev is None else dev):
        _refuse(B.SSM_ERR_UNSUPPORTED, where, name, t)


def _empty(shape, dtype, device, stream):
    """A new tensor in the memory of the stream that will write it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device) if stream else \
            torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _matrix_like(rows, width, ld, dtype, device, stream):
    if ld in (0, width) or rows < 2:
        return _empty((rows, width), dtype, device, stream)
    return _empty((rows, ld), dtype, device, stream)[:, :width]


def _io_of(t, where):
    if t.dtype is torch.bfloat16:
        return B.SSM_BF16
    if t.dtype is torch.float32:
        return B.SSM_F32
    _refuse(B.SSM_ERR_DTYPE, where, "the tensor", t)


def ckpt8_bytes(n_rows, width) -> int:
    """Size of the 8-bit checkpoint of an [n_rows][width] tensor
    (ssm_ckpt8_bytes, without a call into the library)."""
    return n_rows * ((width + 31) // 32) * 33


def ckpt8_empty(n_rows, width, device="cuda", stream=None) -> torch.Tensor:
    """Memory for the 8-bit checkpoint of an [n_rows][width] tensor."""
    return _empty((ckpt8_bytes(n_rows, width),), torch.uint8, device, stream)


def ckpt8_pack(x: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """The 8-bit checkpoint of x [n_rows][width] (f32 or bf16)."""
    where, dev = "ckpt8_pack", _device_of(stream)
    io, (rows, width) = _io_of(x, where), x.shape
    ld = x.stride(0) if rows > 1 else width
    _matrix(where, "x", x, rows, width, ld, x.dtype, dev)
    if out is None:
        out = ckpt8_empty(rows, width, x.device, stream)
    _dense(where, "out", out, ckpt8_bytes(rows, width), torch.uint8, dev)
    B.ssm_ckpt8_pack(x, ld, rows, width, io, out, stream)
    return out


def ckpt8_unpack(ckpt: torch.Tensor, n_rows, width, io="bf16", out=None, stream=None) -> torch.Tensor:
    """The values an 8-bit checkpoint holds, [n_rows][width] in out's type (io
    without out)."""
    where, dev = "ckpt8_unpack", _device_of(stream)
    if out is None:
        _dense(where, "ckpt", ckpt, ckpt8_bytes(n_rows, width), torch.uint8, dev)
        out = _empty((n_rows, width), TORCH_IO[IO_DTYPES[io]], ckpt.device, stream)
        ld = width
    else:
        ld = out.stride(0) if n_rows > 1 else width
        _matrix(where, "out", out, n_rows, width, ld, out.dtype, dev)
        _dense(where, "ckpt", ckpt, ckpt8_bytes(n_rows, width), torch.uint8, dev)
    B.ssm_ckpt8_unpack(ckpt, out, ld, n_rows, width, _io_of(out, where), stream)
    return out


def ckpt8_wgrad_workspace(n_rows, width, n_out, io="bf16", device="cuda", stream=None) -> torch.Tensor:
    n = B.ssm_ckpt8_wgrad_workspace_bytes(n_rows, width, n_out, IO_DTYPES[io])
    return _empty((max(n, 4),), torch.uint8, device, stream)


def ckpt8_wgrad(dy: torch.Tensor, ckpt: torch.Tensor, width, *, dw=None, accumulate=False, ws=None,
                stream=None) -> torch.Tensor:
    """Weight gradient dw [n_out][width] (f32) of out = x W^T from dy
    [n_rows][n_out] and the 8-bit checkpoint of x [n_rows][width]; added to dw
    with accumulate."""
    where, dev = "ckpt8_wgrad", _device_of(stream)
    io, (rows, n_out) = _io_of(dy, where), dy.shape
    ld = dy.stride(0) if rows > 1 else n_out
    _matrix(where, "dy", dy, rows, n_out, ld, dy.dtype, dev)
    _dense(where, "ckpt", ckpt, ckpt8_bytes(rows, width), torch.uint8, dev)
    if dw is None:
        if accumulate:
            raise B.SsmError(B.SSM_ERR_NULL, f"{where}: accumulate without dw")
        dw = _empty((n_out, width), torch.float32, dy.device, stream)
    _dense(where, "dw", dw, n_out * width, torch.float32, dev)
    if ws is None:
        n = B.ssm_ckpt8_wgrad_workspace_bytes(rows, width, n_out, io)
        ws = _empty((n,), torch.uint8, dy.device, stream)
    else:
        _dense(where, "ws", ws, 0, ws.dtype, dev)
    B.ssm_ckpt8_wgrad(dy, ld, ckpt, dw, rows, width, n_out, io, bool(accumulate), ws,
                      ws.numel(), stream)
    return dw


def norm_desc(*, n_rows, width, n_group=1, io="bf16", res="f32", eps=1e-5, res_scale=1.0,
              gate_after=False, ld_x=0, ld_z=0, ld_res=0, ld_out=0) -> B.SsmNormDesc:
    """Descriptor of the two norms.  ld_x, ld_z, ld_res, ld_out: row strides in
    elements (0: width) of y or b, of z, of the residual stream, and of out or
    h; a gradient has its tensor's."""
    def dtype(v):
        return IO_DTYPES[v] if isinstance(v, str) else int(v)

    return B.SsmNormDesc(int(n_rows), int(width), int(n_group), int(ld_x) or int(width),
                         int(ld_z) or int(width), int(ld_res) or int(width),
                         int(ld_out) or int(width), dtype(io), dtype(res), float(eps),
                         float(res_scale), B.SSM_NORM_GATE_AFTER if gate_after else 0, 0)


def norm_bwd_workspace(desc: B.SsmNormDesc, device="cuda", stream=None) -> torch.Tensor:
    n = B.ssm_norm_bwd_workspace_bytes(desc)
    if n == 0:
        raise B.SsmError(B.SSM_ERR_SHAPE, "ssm_norm_bwd_workspace_bytes")
    return _empty((n,), torch.uint8, device, stream)


@dataclass
class NormGatedResult:
    out: torch.Tensor              # [n_rows][width] io
    rstd: Optional[torch.Tensor]   # [n_rows][n_group] f32
    y8: Optional[torch.Tensor]     # 8-bit checkpoints of y, z and out
    z8: Optional[torch.Tensor]
    out8: Optional[torch.Tensor]


def norm_gated_fwd(desc, y, z, w, *, train=False, out=None, rstd=None, y8=None, z8=None, out8=None,
                   stream=None) -> NormGatedResult:
    """The gated norm after the scan (ssm_norm_gated_fwd).  train: also what
    the backward needs, rstd and the 8-bit checkpoints y8 and z8, in new
    tensors where none is given."""
    where, M, W, io = "norm_gated_fwd", desc.n_rows, desc.width, TORCH_IO[desc.io_dtype]
    dev = _device_of(stream)
    _matrix(where, "y", y, M, W, desc.ld_x, io, dev)
    _matrix(where, "z", z, M, W, desc.ld_z, io, dev)
    _dense(where, "w", w, W, torch.float32, dev)
    if out is None:
        out = _matrix_like(M, W, desc.ld_out, io, y.device, stream)
    else:
        _matrix(where, "out", out, M, W, desc.ld_out, io, dev)
    if train:
        rstd = _empty((M, desc.n_group), torch.float32, y.device, stream) if rstd is None else rstd
        y8 = ckpt8_empty(M, W, y.device, stream) if y8 is None else y8
        if z is not None:
            z8 = ckpt8_empty(M, W, y.device, stream) if z8 is None else z8
    _dense(where, "rstd", rstd, M * desc.n_group, torch.float32, dev)
    if y8 is not None or z8 is not None or out8 is not None:
        n = ckpt8_bytes(M, W)
        _dense(where, "y8", y8, n, torch.uint8, dev)
        _dense(where, "z8", z8, n, torch.uint8, dev)
        _dense(where, "out8", out8, n, torch.uint8, dev)
    B.ssm_norm_gated_fwd(desc, y, z, w, out, rstd, y8, z8, out8, stream)
    return NormGatedResult(out, rstd, y8, z8, out8)


@dataclass
class NormGatedGrad:
    d_y: torch.Tensor
    d_z: Optional[torch.Tensor]
    d_w: torch.Tensor


def norm_gated_bwd(desc, dout, w, rstd, *, y=None, z=None, y8=None, z8=None, d_y=None, d_z=None,
                   d_w=None, ws=None, stream=None) -> NormGatedGrad:
    """Backward of ``norm_gated_fwd`` from y and z or their 8-bit checkpoints."""
    where, M, W, io = "norm_gated_bwd", desc.n_rows, desc.width, TORCH_IO[desc.io_dtype]
    dev = _device_of(stream)
    _matrix(where, "dout", dout, M, W, desc.ld_out, io, dev)
    _matrix(where, "y", y, M, W, desc.ld_x, io, dev)
    _matrix(where, "z", z, M, W, desc.ld_z, io, dev)
    _dense(where, "w", w, W, torch.float32, dev)
    _dense(where, "rstd", rstd, M * desc.n_group, torch.float32, dev)
    if y8 is not None or z8 is not None:
        n = ckpt8_bytes(M, W)
        _dense(where, "y8", y8, n, torch.uint8, dev)
        _dense(where, "z8", z8, n, torch.uint8, dev)
    if d_y is None:
        d_y = _matrix_like(M, W, desc.ld_x, io, dout.device, stream)
    else:
        _matrix(where, "d_y", d_y, M, W, desc.ld_x, io, dev)
    if d_z is not None:
        _matrix(where, "d_z", d_z, M, W, desc.ld_z, io, dev)
    elif z is not None or z8 is not None:
        d_z = _matrix_like(M, W, desc.ld_z, io, dout.device, stream)
    if d_w is None:
        d_w = _empty((W,), torch.float32, dout.device, stream)
    else:
        _dense(where, "d_w", d_w, W, torch.float32, dev)
    if ws is None:
        ws = norm_bwd_workspace(desc, dout.device, stream)
    else:
        _dense(where, "ws", ws, 0, ws.dtype, dev)
    B.ssm_norm_gated_bwd(desc, dout, y, z, y8, z8, w, rstd, d_y, d_z, d_w, ws, ws.numel(), stream)
    return NormGatedGrad(d_y, d_z, d_w)


@dataclass
class NormResidualResult:
    r_out: torch.Tensor                # [n_rows][width] residual stream
    h: torch.Tensor                    # [n_rows][width] io
    rstd: Optional[torch.Tensor]       # [n_rows] f32
    rstd_post: Optional[torch.Tensor]  # [n_rows] f32, with w_post
    r8: Optional[torch.Tensor]         # 8-bit checkpoints of r_out, b and h
    b8: Optional[torch.Tensor]
    h8: Optional[torch.Tensor]


def norm_residual_fwd(desc, b, r, w, *, w_post=None, scale=None, train=False, r_out=None, h=None,
                      rstd=None, rstd_post=None, r8=None, b8=None, h8=None,
                      stream=None) -> NormResidualResult:
    """The norm between two blocks (ssm_norm_residual_fwd): the branch b into
    the residual stream r, and the stream's norm for the next block.  train:
    also what the backward needs, rstd, rstd_post and the 8-bit checkpoints r8
    and (with w_post or scale) b8, and h8 for the next projection's weight
    gradient, in new tensors where none is given.  r_out may be r."""
    where, M, W = "norm_residual_fwd", desc.n_rows, desc.width
    dev = _device_of(stream)
    io, res = TORCH_IO[desc.io_dtype], TORCH_IO[desc.res_dtype]
    _matrix(where, "b", b, M, W, desc.ld_x, io, dev)
    _matrix(where, "r", r, M, W, desc.ld_res, res, dev)
    _dense(where, "w", w, W, torch.float32, dev)
    _dense(where, "w_post", w_post, W, torch.float32, dev)
    _dense(where, "scale", scale, W, torch.float32, dev)
    if r_out is None:
        r_out = _matrix_like(M, W, desc.ld_res, res, w.device, stream)
    else:
        _matrix(where, "r_out", r_out, M, W, desc.ld_res, res, dev)
    if h is None:
        h = _matrix_like(M, W, desc.ld_out, io, w.device, stream)
    else:
        _matrix(where, "h", h, M, W, desc.ld_out, io, dev)
    if train:
        rstd = _empty((M,), torch.float32, w.device, stream) if rstd is None else rstd
        if w_post is not None and rstd_post is None:
            rstd_post = _empty((M,), torch.float32, w.device, stream)
        r8 = ckpt8_empty(M, W, w.device, stream) if r8 is None else r8
        h8 = ckpt8_empty(M, W, w.device, stream) if h8 is None else h8
        if (w_post is not None or scale is not None) and b8 is None:
            b8 = ckpt8_empty(M, W, w.device, stream)
    _dense(where, "rstd", rstd, M, torch.float32, dev)
    _dense(where, "rstd_post", rstd_post, M, torch.float32, dev)
    if r8 is not None or b8 is not None or h8 is not None:
        n = ckpt8_bytes(M, W)
        _dense(where, "r8", r8, n, torch.uint8, dev)
        _dense(where, "b8", b8, n, torch.uint8, dev)
        _dense(where, "h8", h8, n, torch.uint8, dev)
    B.ssm_norm_residual_fwd(desc, b, r, w_post, scale, w, r_out, h, rstd, rstd_post, r8, b8, h8,
                            stream)
    return NormResidualResult(r_out, h, rstd, rstd_post, r8, b8, h8)


@dataclass
class NormResidualGrad:
    d_r: torch.Tensor
    d_b: torch.Tensor
    d_w: torch.Tensor
    d_w_post: Optional[torch.Tensor]
    d_scale: Optional[torch.Tensor]


def norm_residual_bwd(desc, dh, w, rstd, *, dr_out=None, r_out=None, r8=None, b=None, b8=None,
                      rstd_post=None, w_post=None, scale=None, d_r=None, d_b=None, d_w=None,
                      d_w_post=None, d_scale=None, ws=None, stream=None) -> NormResidualGrad:
    """Backward of ``norm_residual_fwd`` from r_out or its 8-bit checkpoint
    (and b or its, with w_post or for d_scale).  A scale without b, b8 and
    d_scale is a constant: its gradient is not formed.  d_r may be dr_out."""
    where, M, W = "norm_residual_bwd", desc.n_rows, desc.width
    dev = _device_of(stream)
    io, res = TORCH_IO[desc.io_dtype], TORCH_IO[desc.res_dtype]
    _matrix(where, "dh", dh, M, W, desc.ld_out, io, dev)
    _matrix(where, "dr_out", dr_out, M, W, desc.ld_res, res, dev)
    _matrix(where, "r_out", r_out, M, W, desc.ld_res, res, dev)
    _matrix(where, "b", b, M, W, desc.ld_x, io, dev)
    _dense(where, "w", w, W, torch.float32, dev)
    _dense(where, "w_post", w_post, W, torch.float32, dev)
    _dense(where, "scale", scale, W, torch.float32, dev)
    _dense(where, "rstd", rstd, M, torch.float32, dev)
    _dense(where, "rstd_post", rstd_post, M, torch.float32, dev)
    if r8 is not None or b8 is not None:
        n = ckpt8_bytes(M, W)
        _dense(where, "r8", r8, n, torch.uint8, dev)
        _dense(where, "b8", b8, n, torch.uint8, dev)
    if d_r is None:
        d_r = _matrix_like(M, W, desc.ld_res, res, dh.device, stream)
    else:
        _matrix(where, "d_r", d_r, M, W, desc.ld_res, res, dev)
    if d_b is None:
        d_b = _matrix_like(M, W, desc.ld_x, io, dh.device, stream)
    else:
        _matrix(where, "d_b", d_b, M, W, desc.ld_x, io, dev)
    if d_w is None:
        d_w = _empty((W,), torch.float32, dh.device, stream)
    if w_post is not None and d_w_post is None:
        d_w_post = _empty((W,), torch.float32, dh.device, stream)
    if scale is not None and d_scale is None and (b is not None or b8 is not None):
        d_scale = _empty((W,), torch.float32, dh.device, stream)
    _dense(where, "d_w", d_w, W, torch.float32, dev)
    _dense(where, "d_w_post", d_w_post, W, torch.float32, dev)
    _dense(where, "d_scale", d_scale, W, torch.float32, dev)
    if ws is None:
        ws = norm_bwd_workspace(desc, dh.device, stream)
    else:
        _dense(where, "ws", ws, 0, ws.dtype, dev)
    B.ssm_norm_residual_bwd(desc, dh, dr_out, r_out, r8, b, b8, w_post, scale, w, rstd, rstd_post,
                            d_r, d_b, d_w, d_w_post, d_scale, ws, ws.numel(), stream)
    return NormResidualGrad(d_r, d_b, d_w, d_w_post, d_scale)


# ---- the loss over the vocabulary ----
#
# As above: [n_rows][width] and [n_vocab][width] matrices with a contiguous last
# axis, everything checked here that the C ABI cannot see, on the call's device.


def vocab_desc(*, n_rows, width, n_vocab, n_top=0, io="bf16", dw="f32", scale=1.0, top_scale=1.0,
               ld_h=0, ld_w=0, accumulate=False) -> B.SsmVocabDesc:
    """Descriptor of the losses over a vocabulary.  n_top: the teacher's entries
    a row (0: cross entropy).  dw: type of d_w, f32 or io's.  ld_h, ld_w: row
    strides in elements (0: width) of h and d_h, and of w and d_w.  accumulate:
    the backward adds to d_w."""
    def dtype(v):
        return IO_DTYPES[v] if isinstance(v, str) else int(v)

    return B.SsmVocabDesc(int(n_rows), int(width), int(n_vocab), int(n_top), int(ld_h) or int(width),
                          int(ld_w) or int(width), dtype(io), dtype(dw), float(scale),
                          float(top_scale), B.SSM_VOCAB_ACCUMULATE if accumulate else 0, 0)


def vocab_workspace(desc: B.SsmVocabDesc, backward: bool, device="cuda", stream=None) -> torch.Tensor:
    """Workspace of a forward, or of a backward (which serves the forward too)."""
    n = B.ssm_vocab_workspace_bytes(desc, int(backward))
    if n == 0:
        raise B.SsmError(B.SSM_ERR_SHAPE, "ssm_vocab_workspace_bytes")
    return _empty((n,), torch.uint8, device, stream)


@dataclass
class VocabLoss:
    loss: torch.Tensor             # [n_rows] f32
    lse: torch.Tensor              # [n_rows] f32
    logq: Optional[torch.Tensor]   # [n_rows][n_top] f32 (distillation)


@dataclass
class VocabGrad:
    d_h: Optional[torch.Tensor]    # [n_rows][width] io
    d_w: Optional[torch.Tensor]    # [n_vocab][width]


def _vocab_inputs(where, desc, h, w, dev):
    _matrix(where, "h", h, desc.n_rows, desc.width, desc.ld_h, TORCH_IO[desc.io_dtype], dev)
    _matrix(where, "w", w, desc.n_vocab, desc.width, desc.ld_w, TORCH_IO[desc.io_dtype], dev)


def _vocab_entries(where, name, t, desc, dtype, dev):
    """[n_rows][n_top], dense."""
    if t is not None and t.shape != (desc.n_rows, desc.n_top):
        _refuse(B.SSM_ERR_SHAPE, where, name, t)
    _dense(where, name, t, desc.n_rows * desc.n_top, dtype, dev)


def _vocab_fwd(where, desc, h, w, loss, lse, err, ws, dev, stream):
    _vocab_inputs(where, desc, h, w, dev)
    M = desc.n_rows
    loss = _empty((M,), torch.float32, w.device, stream) if loss is None else loss
    lse = _empty((M,), torch.float32, w.device, stream) if lse is None else lse
    _dense(where, "loss", loss, M, torch.float32, dev)
    _dense(where, "lse", lse, M, torch.float32, dev)
    if err is not None:
        _dense(where, "err", err, 1, torch.int32, dev)
    if ws is None:
        ws = vocab_workspace(desc, False, w.device, stream)
    else:
        _dense(where, "ws", ws, 0, ws.dtype, dev)
    return loss, lse, ws


def _vocab_bwd(where, desc, h, w, lse, d_loss, d_lse, d_h, d_w, want_h, want_w, ws, dev, stream):
    _vocab_inputs(where, desc, h, w, dev)
    M, io, dw = desc.n_rows, TORCH_IO[desc.io_dtype], TORCH_IO[desc.dw_dtype]
    _dense(where, "lse", lse, M, torch.float32, dev)
    _dense(where, "d_loss", d_loss, M, torch.float32, dev)
    _dense(where, "d_lse", d_lse, M, torch.float32, dev)
    if d_h is None and want_h:
        d_h = _matrix_like(M, desc.width, desc.ld_h, io, w.device, stream)
    _matrix(where, "d_h", d_h, M, desc.width, desc.ld_h, io, dev)
    if d_w is None and want_w:
        if desc.flags & B.SSM_VOCAB_ACCUMULATE:
            raise B.SsmError(B.SSM_ERR_NULL, f"{where}: accumulate without d_w")
        d_w = _matrix_like(desc.n_vocab, desc.width, desc.ld_w, dw, w.device, stream)
    _matrix(where, "d_w", d_w, desc.n_vocab, desc.width, desc.ld_w, dw, dev)
    if ws is None:
        ws = vocab_workspace(desc, True, w.device, stream)
    else:
        _dense(where, "ws", ws, 0, ws.dtype, dev)
    return d_h, d_w, ws


def vocab_ce_fwd(desc, h, w, target, *, loss=None, lse=None, err=None, ws=None, stream=None) -> VocabLoss:
    """Softmax cross entropy of scale * h w^T against target [n_rows] int32
    (ssm_vocab_ce_fwd): a loss a row, 0 where the target is negative."""
    where, dev = "vocab_ce_fwd", _device_of(stream)
    loss, lse, ws = _vocab_fwd(where, desc, h, w, loss, lse, err, ws, dev, stream)
    _dense(where, "target", target, desc.n_rows, torch.int32, dev)
    B.ssm_vocab_ce_fwd(desc, h, w, target, loss, lse, err, ws, ws.numel(), stream)
    return VocabLoss(loss, lse, None)


def vocab_ce_bwd(desc, h, w, target, loss, lse, d_loss, *, d_lse=None, d_h=None, d_w=None, want_h=True,
                 want_w=True, ws=None, stream=None) -> VocabGrad:
    """Backward of ``vocab_ce_fwd`` from its loss and lse.  want_h, want_w: form
    the gradient although no tensor is given for it."""
    where, dev = "vocab_ce_bwd", _device_of(stream)
    _dense(where, "target", target, desc.n_rows, torch.int32, dev)
    _dense(where, "loss", loss, desc.n_rows, torch.float32, dev)
    d_h, d_w, ws = _vocab_bwd(where, desc, h, w, lse, d_loss, d_lse, d_h, d_w, want_h, want_w, ws, dev,
                              stream)
    B.ssm_vocab_ce_bwd(desc, h, w, target, loss, lse, d_loss, d_lse, d_h, d_w, ws, ws.numel(), stream)
    return VocabGrad(d_h, d_w)


def vocab_kd_fwd(desc, h, w, top_id, top_logit, *, top_lse=None, loss=None, lse=None, logq=None, err=None,
                 ws=None, stream=None) -> VocabLoss:
    """Distillation from a teacher's top logits [n_rows][n_top] f32 at top_id
    int32 (ssm_vocab_kd_fwd).  An id < 0 or a logit of -inf is no entry."""
    where, dev = "vocab_kd_fwd", _device_of(stream)
    loss, lse, ws = _vocab_fwd(where, desc, h, w, loss, lse, err, ws, dev, stream)
    if logq is None:
        logq = _empty((desc.n_rows, desc.n_top), torch.float32, w.device, stream)
    _vocab_entries(where, "top_id", top_id, desc, torch.int32, dev)
    _vocab_entries(where, "top_logit", top_logit, desc, torch.float32, dev)
    _vocab_entries(where, "logq", logq, desc, torch.float32, dev)
    _dense(where, "top_lse", top_lse, desc.n_rows, torch.float32, dev)
    B.ssm_vocab_kd_fwd(desc, h, w, top_id, top_logit, top_lse, loss, lse, logq, err, ws, ws.numel(), stream)
    return VocabLoss(loss, lse, logq)


def vocab_kd_bwd(desc, h, w, top_id, top_logit, logq, lse, d_loss, *, top_lse=None, d_lse=None, d_h=None,
                 d_w=None, want_h=True, want_w=True, ws=None, stream=None) -> VocabGrad:
    """Backward of ``vocab_kd_fwd`` from its logq and lse."""
    where, dev = "vocab_kd_bwd", _device_of(stream)
    _vocab_entries(where, "top_id", top_id, desc, torch.int32, dev)
    _vocab_entries(where, "top_logit", top_logit, desc, torch.float32, dev)
    _vocab_entries(where, "logq", logq, desc, torch.float32, dev)
    _dense(where, "top_lse", top_lse, desc.n_rows, torch.float32, dev)
    d_h, d_w, ws = _vocab_bwd(where, desc, h, w, lse, d_loss, d_lse, d_h, d_w, want_h, want_w, ws, dev,
                              stream)
    B.ssm_vocab_kd_bwd(desc, h, w, top_id, top_logit, top_lse, logq, lse, d_loss, d_lse, d_h, d_w, ws,
                       ws.numel(), stream)
    return VocabGrad(d_h, d_w)
