"""Python binding of the operators around the scan: the gated recurrence, the
short causal convolution and the token embedding.

Argument marshalling only, as in ``lrscan`` (which re-exports these
functions); the arithmetic runs in the library's CUDA kernels.  [B, T, D]
tensors here need contiguous channels only: a slice of a wider projection is
read, and a gradient written into one, in place.
"""
from __future__ import annotations

import ctypes

import torch

from . import lrscan as _l

SAVE_EVERY = 16   # tokens between the states that the gated recurrence saves

_raw_stream = torch._C._cuda_getCurrentRawStream


class Rows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_t", ctypes.c_int64)]


_RP, _P, _I64, _F, _INT = ctypes.POINTER(Rows), ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int
_SP, _OP = ctypes.POINTER(_l.State), ctypes.POINTER(_l.Opts)

EXPORTS = {
    "lrscan_fwd_gates": ([_RP, _RP, _RP, _P, _F, _RP, _P, _P, _SP, _I64, _I64, _I64, _INT, _P, _OP], _INT),
    "lrscan_bwd_gates": ([_RP, _RP, _RP, _P, _F, _P, _RP, _RP, _RP, _RP, _P, _SP, _I64, _I64, _I64, _INT, _P, _OP], _INT),
    "lrscan_step_gates": ([_RP, _RP, _RP, _P, _F, _P, _P, _RP, _I64, _I64, _I64, _INT, _P], _INT),
    "lrscan_gates_workspace_bytes": ([_I64, _I64, _I64, _INT, _INT], ctypes.c_size_t),
    "lrscan_fwd_conv": ([_RP, _P, _P, _INT, _P, _P, _RP, _P, _I64, _I64, _I64, _INT, _P], _INT),
    "lrscan_bwd_conv": ([_RP, _P, _INT, _P, _P, _RP, _P, _RP, _P, _P, _P, _I64, _I64, _I64, _INT, _P, _OP], _INT),
    "lrscan_conv_workspace_bytes": ([_I64, _I64, _I64, _INT], ctypes.c_size_t),
    "lrscan_step_conv": ([_RP, _P, _P, _INT, _P, _P, _RP, _I64, _I64, _I64, _INT, _P], _INT),
    "lrscan_fwd_embed": ([_P, _INT, _P, _INT, _F, _P, _INT, _I64, _I64, _I64, _P], _INT),
    "lrscan_bwd_embed": ([_P, _INT, _P, _INT, _F, _P, _INT, _INT, _I64, _I64, _I64, _P, _OP], _INT),
    "lrscan_embed_workspace_bytes": ([_I64, _I64, _I64], ctypes.c_size_t),
}
_l.EXPORTS.update(EXPORTS)


class _On:
    """The tensors' device made current for the call, where it is not."""

    def __init__(self, device):
        self.guard = None if device.index == torch.cuda.current_device() else torch.cuda.device(device)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _stream(stream, device) -> int:
    return _raw_stream(device.index) if stream is None else stream.cuda_stream


def _rows(name, t, shape, dtype, device):
    """A tensor with contiguous channels, as the library takes it ([B, D]: one token)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} is on {t.device}, expected a CUDA device ({device})")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    st = t.stride()
    if shape[-1] > 1 and st[-1] != 1:
        raise ValueError(f"{name} must have contiguous channels (stride 1 in the last dimension)")
    return Rows(t.data_ptr(), st[0], st[1] if len(st) == 3 else 0)


def _dense(name, t, shape, dtype, device):
    """Pointer of a contiguous tensor, or None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device or t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _tokens(x, name="x"):
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.ndim != 3:
        raise ValueError(f"{name} must be a [B, T, D] tensor")
    if not x.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    return x.shape, _l._dtype_code(x)


def _new(x, shape=None, dtype=None):
    return torch.empty(x.shape if shape is None else shape, device=x.device, dtype=dtype or x.dtype)


def _saved_shape(B, T, D):
    return torch.Size((B, (T + SAVE_EVERY - 1) // SAVE_EVERY, D))


# ---------------------------------------------------------------------------
# gated recurrence
# ---------------------------------------------------------------------------
def lrscan_fwd_gates(r, i, x, lam, *, c: float = 8.0, h0=None, segment_pos=None, out=None, last=None, saved=None,
                     want_saved: bool = False, workspace=None, stream=None):
    """Gated recurrence h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t with
    a_t = exp(-c softplus(lam) sigmoid(r_t)), from the fp32 [B, D] state h0,
    restarting (a_t = 0) where the int32 [B, T] segment_pos is 0; r, i, x
    [B, T, D], lam fp32 [D].  Returns (out, last, saved): the states in the
    storage dtype, the fp32 [B, D] final state, and (want_saved) the fp32 states
    before tokens 0, 16, 32, ... that the backward needs, else None."""
    shape, code = _tokens(x)
    B, T, D = shape
    dev, dt = x.device, x.dtype
    out = _new(x) if out is None else out
    last = _new(x, (B, D), torch.float32) if last is None else last
    if saved is None and want_saved:
        saved = _new(x, _saved_shape(B, T, D), torch.float32)
    rr, ri, rx = (_rows(n, t, shape, dt, dev) for n, t in (("r", r), ("i", i), ("x", x)))
    ro = _rows("out", out, shape, dt, dev)
    bd = torch.Size((B, D))
    st = _l.State()
    st.h0 = _dense("h0", h0, bd, torch.float32, dev)
    st.segment_pos = _dense("segment_pos", segment_pos, shape[:2], torch.int32, dev)
    lp = _dense("lam", lam, shape[2:], torch.float32, dev)
    with _On(dev):
        o = None if workspace is None else _l._opts(None, None, None, workspace)
        rc = _l.lib().lrscan_fwd_gates(rr, ri, rx, lp, c, ro, _dense("last", last, bd, torch.float32, dev),
                                       _dense("saved", saved, _saved_shape(B, T, D), torch.float32, dev), st, B, T, D,
                                       code, _stream(stream, dev), o)
    _l._check(rc, "lrscan_fwd_gates")
    return out, last, saved


def lrscan_bwd_gates(r, i, x, lam, saved, grad_out, *, c: float = 8.0, segment_pos=None, grad_last=None, grad_r=None,
                     grad_i=None, grad_x=None, grad_lam=None, grad_h0=None, want_grad_h0: bool = True, workspace=None,
                     stream=None):
    """Reverse of :func:`lrscan_fwd_gates` for the loss sum(grad_out * out) +
    sum(grad_last * last), from the states it saved; returns (grad_r, grad_i,
    grad_x, grad_lam, grad_h0) (grad_h0 None when not wanted)."""
    shape, code = _tokens(x)
    B, T, D = shape
    dev, dt = x.device, x.dtype
    grad_r = _new(x) if grad_r is None else grad_r
    grad_i = _new(x) if grad_i is None else grad_i
    grad_x = _new(x) if grad_x is None else grad_x
    grad_lam = _new(x, (D,), torch.float32) if grad_lam is None else grad_lam
    bd = torch.Size((B, D))
    if grad_h0 is None and want_grad_h0:
        grad_h0 = _new(x, bd, torch.float32)
    rr, ri, rx, rg, r0, r1, r2 = (
        _rows(n, t, shape, dt, dev) for n, t in (("r", r), ("i", i), ("x", x), ("grad_out", grad_out),
                                                 ("grad_r", grad_r), ("grad_i", grad_i), ("grad_x", grad_x)))
    st = _l.State()
    st.segment_pos = _dense("segment_pos", segment_pos, shape[:2], torch.int32, dev)
    st.grad_last = _dense("grad_last", grad_last, bd, torch.float32, dev)
    st.grad_h0 = _dense("grad_h0", grad_h0, bd, torch.float32, dev)
    lp = _dense("lam", lam, shape[2:], torch.float32, dev)
    sp = _dense("saved", saved, _saved_shape(B, T, D), torch.float32, dev)
    with _On(dev):
        o = None if workspace is None else _l._opts(None, None, None, workspace)
        rc = _l.lib().lrscan_bwd_gates(rr, ri, rx, lp, c, sp, rg, r0, r1, r2,
                                       _dense("grad_lam", grad_lam, shape[2:], torch.float32, dev), st, B, T, D, code,
                                       _stream(stream, dev), o)
    _l._check(rc, "lrscan_bwd_gates")
    return grad_r, grad_i, grad_x, grad_lam, grad_h0


def lrscan_step_gates(r, i, x, lam, state, *, slots=None, c: float = 8.0, out=None, stream=None):
    """One token of each of B requests: r, i, x [B, D]; request b's state is row
    slots[b] (int32 [B]; row b without slots) of the fp32 pool state [S, D],
    updated in place.  Returns out [B, D]; a negative slot gives zeros."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.ndim != 2 or not x.is_cuda:
        raise ValueError("x must be a CUDA [B, D] tensor")
    shape, code, dev, dt = x.shape, _l._dtype_code(x), x.device, x.dtype
    B, D = shape
    if state.ndim != 2:
        raise ValueError("state must be a [S, D] tensor")
    S = state.shape[0]
    out = _new(x) if out is None else out
    rr, ri, rx, ro = (_rows("r", r, shape, dt, dev), _rows("i", i, shape, dt, dev), _rows("x", x, shape, dt, dev),
                      _rows("out", out, shape, dt, dev))
    lp = _dense("lam", lam, shape[1:], torch.float32, dev)
    sp = _dense("state", state, torch.Size((S, D)), torch.float32, dev)
    tp = _dense("slots", slots, shape[:1], torch.int32, dev)
    with _On(dev):
        rc = _l.lib().lrscan_step_gates(rr, ri, rx, lp, c, sp, tp, ro, B, S, D, code, _stream(stream, dev))
    _l._check(rc, "lrscan_step_gates")
    return out


def lrscan_gates_workspace_bytes(B: int, T: int, D: int, dtype="f32", direction: str = "fwd") -> int:
    """Bytes of device scratch of a gated-recurrence call."""
    code = {"f32": _l.F32, "bf16": _l.BF16}.get(dtype) if isinstance(dtype, str) else _l._DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {dtype}")
    return _l.lib().lrscan_gates_workspace_bytes(B, T, D, code, 0 if direction == "fwd" else 1)


class GateScan(torch.autograd.Function):
    """Autograd wrapper of the gated recurrence: (out, last) = scan(r, i, x, lam,
    h0, segment_pos); gradients flow to r, i, x, lam and h0 from both outputs."""

    @staticmethod
    def forward(ctx, r, i, x, lam, h0, segment_pos, c=8.0):
        r, i, x = (t if t.stride(-1) == 1 else t.contiguous() for t in (r, i, x))
        lam = lam.contiguous()
        h0 = h0.contiguous() if h0 is not None else None
        seg = segment_pos.contiguous() if segment_pos is not None else None
        out, last, saved = lrscan_fwd_gates(r, i, x, lam, c=c, h0=h0, segment_pos=seg, want_saved=True)
        ctx.save_for_backward(r, i, x, lam, saved, seg)
        ctx.c, ctx.has_h0 = c, h0 is not None
        return out, last

    @staticmethod
    def backward(ctx, grad_out, grad_last):
        r, i, x, lam, saved, seg = ctx.saved_tensors
        grad_out = torch.zeros_like(x) if grad_out is None else grad_out
        grad_out = grad_out if grad_out.stride(-1) == 1 else grad_out.contiguous()
        g = lrscan_bwd_gates(r, i, x, lam, saved, grad_out, c=ctx.c, segment_pos=seg, want_grad_h0=ctx.has_h0,
                             grad_last=grad_last.contiguous() if grad_last is not None else None)
        return (*g, None, None)


def gate_scan(r, i, x, lam, h0=None, segment_pos=None, c: float = 8.0):
    """Differentiable gated recurrence; returns (out, last) with last fp32 [B, D]."""
    return GateScan.apply(r, i, x, lam, h0, segment_pos, c)


# ---------------------------------------------------------------------------
# causal convolution
# ---------------------------------------------------------------------------
def _taps(w, D):
    if not isinstance(w, torch.Tensor):
        raise TypeError("w must be a torch.Tensor")
    if w.ndim != 2 or w.shape[0] != D:
        raise ValueError(f"w must be a [D, K] tensor, D = {D}; got {tuple(w.shape)}")
    return w.shape[1]


def lrscan_fwd_conv(x, w, bias=None, *, x0=None, segment_pos=None, out=None, last=None, want_last: bool = False,
                    stream=None):
    """Causal convolution of each channel, out_t = bias + sum_k w[:, K-1-k] x_{t-k}
    within a segment; x [B, T, D], w fp32 [D, K] (K = 2 to 8), bias fp32 [D], x0
    [B, K-1, D] the tokens before token 0 (zeros without it), segments starting
    where the int32 [B, T] segment_pos is 0.  Returns (out, last): last
    (want_last) the last K-1 tokens [B, K-1, D], the next call's x0, else None."""
    shape, code = _tokens(x)
    B, T, D = shape
    dev, dt = x.device, x.dtype
    K = _taps(w, D)
    window = torch.Size((B, K - 1, D))
    out = _new(x) if out is None else out
    if last is None and want_last:
        last = _new(x, window)
    rx, ro = _rows("x", x, shape, dt, dev), _rows("out", out, shape, dt, dev)
    with _On(dev):
        rc = _l.lib().lrscan_fwd_conv(rx, _dense("w", w, w.shape, torch.float32, dev),
                                      _dense("bias", bias, shape[2:], torch.float32, dev), K,
                                      _dense("x0", x0, window, dt, dev),
                                      _dense("segment_pos", segment_pos, shape[:2], torch.int32, dev), ro,
                                      _dense("last", last, window, dt, dev), B, T, D, code, _stream(stream, dev))
    _l._check(rc, "lrscan_fwd_conv")
    return out, last


def lrscan_bwd_conv(x, w, grad_out, *, x0=None, segment_pos=None, grad_last=None, grad_x=None, grad_w=None,
                    grad_bias=None, grad_x0=None, want_grad_x0: bool = False, workspace=None, stream=None):
    """Reverse of :func:`lrscan_fwd_conv` for the loss sum(grad_out * out) +
    sum(grad_last * last); returns (grad_x, grad_w, grad_bias, grad_x0), the
    sums in fp32 (grad_x0 None when not wanted)."""
    shape, code = _tokens(x)
    B, T, D = shape
    dev, dt = x.device, x.dtype
    K = _taps(w, D)
    window = torch.Size((B, K - 1, D))
    grad_x = _new(x) if grad_x is None else grad_x
    grad_w = _new(w) if grad_w is None else grad_w
    grad_bias = _new(x, (D,), torch.float32) if grad_bias is None else grad_bias
    if grad_x0 is None and want_grad_x0:
        grad_x0 = _new(x, window)
    rx, rg, ro = _rows("x", x, shape, dt, dev), _rows("grad_out", grad_out, shape, dt, dev), _rows("grad_x", grad_x, shape,
                                                                                                dt, dev)
    with _On(dev):
        o = None if workspace is None else _l._opts(None, None, None, workspace)
        rc = _l.lib().lrscan_bwd_conv(rx, _dense("w", w, w.shape, torch.float32, dev), K,
                                      _dense("x0", x0, window, dt, dev),
                                      _dense("segment_pos", segment_pos, shape[:2], torch.int32, dev), rg,
                                      _dense("grad_last", grad_last, window, dt, dev), ro,
                                      _dense("grad_w", grad_w, w.shape, torch.float32, dev),
                                      _dense("grad_bias", grad_bias, shape[2:], torch.float32, dev),
                                      _dense("grad_x0", grad_x0, window, dt, dev), B, T, D, code, _stream(stream, dev), o)
    _l._check(rc, "lrscan_bwd_conv")
    return grad_x, grad_w, grad_bias, grad_x0


def lrscan_step_conv(x, w, state, *, bias=None, slots=None, out=None, stream=None):
    """One token of each of B requests: x [B, D]; request b's window is row
    slots[b] (int32 [B]; row b without slots) of the pool state [S, K-1, D] in
    x's dtype, updated in place.  Returns out [B, D]; a negative slot gives zeros."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.ndim != 2 or not x.is_cuda:
        raise ValueError("x must be a CUDA [B, D] tensor")
    shape, code, dev, dt = x.shape, _l._dtype_code(x), x.device, x.dtype
    B, D = shape
    K = _taps(w, D)
    if state.ndim != 3:
        raise ValueError("state must be a [S, K-1, D] tensor")
    S = state.shape[0]
    out = _new(x) if out is None else out
    rx, ro = _rows("x", x, shape, dt, dev), _rows("out", out, shape, dt, dev)
    with _On(dev):
        rc = _l.lib().lrscan_step_conv(rx, _dense("w", w, w.shape, torch.float32, dev),
                                       _dense("bias", bias, shape[1:], torch.float32, dev), K,
                                       _dense("state", state, torch.Size((S, K - 1, D)), dt, dev),
                                       _dense("slots", slots, shape[:1], torch.int32, dev), ro, B, S, D, code,
                                       _stream(stream, dev))
    _l._check(rc, "lrscan_step_conv")
    return out


def lrscan_conv_workspace_bytes(B: int, T: int, D: int, K: int) -> int:
    """Bytes of device scratch of :func:`lrscan_bwd_conv`."""
    return _l.lib().lrscan_conv_workspace_bytes(B, T, D, K)


class CausalConv(torch.autograd.Function):
    """Autograd wrapper of the causal convolution: (out, last) = conv(x, w, bias,
    x0, segment_pos); gradients flow to x, w, bias and x0 from both outputs."""

    @staticmethod
    def forward(ctx, x, w, bias, x0, segment_pos):
        x = x if x.stride(-1) == 1 else x.contiguous()
        w = w.contiguous()
        x0 = x0.contiguous() if x0 is not None else None
        seg = segment_pos.contiguous() if segment_pos is not None else None
        out, last = lrscan_fwd_conv(x, w, bias.contiguous() if bias is not None else None, x0=x0, segment_pos=seg,
                                    want_last=True)
        ctx.save_for_backward(x, w, x0, seg)
        ctx.has_bias = bias is not None
        return out, last

    @staticmethod
    def backward(ctx, grad_out, grad_last):
        x, w, x0, seg = ctx.saved_tensors
        grad_out = torch.zeros_like(x) if grad_out is None else grad_out
        grad_out = grad_out if grad_out.stride(-1) == 1 else grad_out.contiguous()
        gx, gw, gb, g0 = lrscan_bwd_conv(x, w, grad_out, x0=x0, segment_pos=seg, want_grad_x0=x0 is not None,
                                         grad_last=grad_last.contiguous() if grad_last is not None else None)
        return gx, gw, gb if ctx.has_bias else None, g0, None


def causal_conv(x, w, bias=None, x0=None, segment_pos=None):
    """Differentiable causal convolution of each channel; returns (out, last)."""
    return CausalConv.apply(x, w, bias, x0, segment_pos)


# ---------------------------------------------------------------------------
# token embedding
# ---------------------------------------------------------------------------
_ID_BYTES = {torch.int32: 4, torch.int64: 8}


def _ids(ids, device):
    if not isinstance(ids, torch.Tensor):
        raise TypeError("ids must be a torch.Tensor")
    if ids.dtype not in _ID_BYTES:
        raise ValueError(f"ids must be int32 or int64, got {ids.dtype}")
    if ids.device != device or not ids.is_cuda:
        raise ValueError(f"ids is on {ids.device}, expected a CUDA device ({device})")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    return ids.data_ptr(), _ID_BYTES[ids.dtype]


def _code(dtype):
    if dtype not in _l._DTYPES:
        raise ValueError(f"unsupported dtype {dtype}; lrscan takes float32 or bfloat16 storage")
    return _l._DTYPES[dtype]


def lrscan_fwd_embed(ids, weight, *, scale: float = 1.0, dtype=None, out=None, stream=None):
    """Rows scale * weight[ids] of the table weight [V, D]; ids int32 or int64 of
    any shape (a negative id gives zeros); dtype is the result's (weight's
    without it).  Returns [*ids.shape, D]."""
    if not isinstance(weight, torch.Tensor):
        raise TypeError("weight must be a torch.Tensor")
    if weight.ndim != 2:
        raise ValueError("weight must be a [V, D] tensor")
    dev = weight.device
    ip, size = _ids(ids, dev)
    V, D = weight.shape
    dtype = (weight.dtype if dtype is None else dtype) if out is None else out.dtype
    shape = torch.Size((*ids.shape, D))
    out = _new(weight, shape, dtype) if out is None else out
    wc, oc = _code(weight.dtype), _code(dtype)
    wp, op = _dense("weight", weight, weight.shape, weight.dtype, dev), _dense("out", out, shape, dtype, dev)
    with _On(dev):
        rc = _l.lib().lrscan_fwd_embed(ip, size, wp, wc, scale, op, oc, ids.numel(), V, D, _stream(stream, dev))
    _l._check(rc, "lrscan_fwd_embed")
    return out


def lrscan_bwd_embed(ids, grad_out, V: int, *, scale: float = 1.0, dtype=None, grad_weight=None,
                     accumulate: bool = False, workspace=None, stream=None):
    """Gradient [V, D] of the table of :func:`lrscan_fwd_embed`: scale times the
    sum of grad_out over each id's tokens, in fp32 and in a fixed order; dtype is
    the gradient's (fp32 without it); accumulate adds it to grad_weight."""
    if not isinstance(grad_out, torch.Tensor):
        raise TypeError("grad_out must be a torch.Tensor")
    dev = grad_out.device
    ip, size = _ids(ids, dev)
    if grad_out.ndim != ids.ndim + 1 or grad_out.shape[:-1] != ids.shape:
        raise ValueError(f"grad_out must be [*ids.shape, D]; got {tuple(grad_out.shape)} for ids {tuple(ids.shape)}")
    if accumulate and grad_weight is None:
        raise ValueError("accumulate needs grad_weight")
    D = grad_out.shape[-1]
    shape = torch.Size((V, D))
    dtype = (torch.float32 if dtype is None else dtype) if grad_weight is None else grad_weight.dtype
    grad_weight = _new(grad_out, shape, dtype) if grad_weight is None else grad_weight
    gc, wc = _code(grad_out.dtype), _code(dtype)
    gp = _dense("grad_out", grad_out, grad_out.shape, grad_out.dtype, dev)
    wp = _dense("grad_weight", grad_weight, shape, dtype, dev)
    with _On(dev):
        o = None if workspace is None else _l._opts(None, None, None, workspace)
        rc = _l.lib().lrscan_bwd_embed(ip, size, gp, gc, scale, wp, wc, int(accumulate), ids.numel(), V, D,
                                       _stream(stream, dev), o)
    _l._check(rc, "lrscan_bwd_embed")
    return grad_weight


def lrscan_embed_workspace_bytes(N: int, V: int, D: int) -> int:
    """Bytes of device scratch of :func:`lrscan_bwd_embed`."""
    return _l.lib().lrscan_embed_workspace_bytes(N, V, D)


class Embed(torch.autograd.Function):
    """Autograd wrapper of the token embedding; the gradient has weight's dtype."""

    @staticmethod
    def forward(ctx, ids, weight, scale=1.0, dtype=None):
        ids, weight = ids.contiguous(), weight.contiguous()
        ctx.save_for_backward(ids)
        ctx.scale, ctx.V, ctx.dtype = scale, weight.shape[0], weight.dtype
        return lrscan_fwd_embed(ids, weight, scale=scale, dtype=dtype)

    @staticmethod
    def backward(ctx, grad_out):
        (ids,) = ctx.saved_tensors
        return None, lrscan_bwd_embed(ids, grad_out.contiguous(), ctx.V, scale=ctx.scale, dtype=ctx.dtype), None, None


def embed(ids, weight, scale: float = 1.0, dtype=None):
    """Differentiable lookup scale * weight[ids]; returns [*ids.shape, D]."""
    return Embed.apply(ids, weight, scale, dtype)
