"""The operators around the layer: attention over key ranges with its
gradients, rotary positions, and the norms before and after a block fused
with its gate and residual (``include/httm.h`` defines each).

The functions mirror the C calls: torch tensors become device pointers and
strides, a non-OK status becomes an :class:`~.binding.HttmError`, and there is
no fallback.  Tensors may lie on any one device: the call runs there, on
``stream`` or that device's current stream.  Outputs and workspaces that are
not passed in are allocated with torch on that stream.  Nothing here keeps
state between calls, and no function records an autograd graph: forward and
backward are separate calls, and a tensor that requires grad is refused
unless grad mode is off.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass

import torch

from .binding import HTTM_BF16, HTTM_F32, HttmError, _check, load_library  # noqa: F401

HTTM_ROTARY_HALF, HTTM_ROTARY_PAIRS = 0, 1
HTTM_NORM_NONE, HTTM_NORM_LAYER, HTTM_NORM_RMS = 0, 1, 2

_I32, _I64, _F32, _PTR = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class httm_view(ctypes.Structure):
    _fields_ = [("data", _PTR), ("batch", _I64), ("head", _I64), ("token", _I64)]


class httm_attention(ctypes.Structure):
    _fields_ = [(n, _I32) for n in ("batch", "heads", "kv_heads", "q_len", "kv_len", "d_head", "dtype")] + \
        [("softmax_scale", _F32), ("key_begin", _PTR), ("key_end", _PTR)]


class httm_rotary_cfg(ctypes.Structure):
    _fields_ = [(n, _I32) for n in ("batch", "tokens", "heads", "kv_heads", "d_head", "dtype", "axes", "pairs",
                                    "layout", "inverse")] + \
        [("factor", _F32), ("positions", _PTR), ("position_batch", _I64), ("freqs", _PTR)]


class httm_norm_cfg(ctypes.Structure):
    _fields_ = [("rows", _I64)] + [(n, _I32) for n in ("channels", "stream_dtype", "branch_dtype", "post", "pre",
                                                       "gates")] + \
        [(n, _F32) for n in ("post_eps", "pre_eps", "residual_scale")]


class httm_rows(ctypes.Structure):
    _fields_ = [("data", _PTR), ("row", _I64)]


_PARAMS = ("gate", "post_weight", "post_bias", "pre_weight", "pre_bias")


class httm_norm_weights(ctypes.Structure):
    _fields_ = [(n, _PTR) for n in _PARAMS]


class httm_norm_grads(ctypes.Structure):
    _fields_ = [(n, _PTR) for n in _PARAMS]


_DTYPES = {torch.bfloat16: HTTM_BF16, torch.float32: HTTM_F32}


def _ref(s):
    return None if s is None else ctypes.byref(s)


def _data(t):
    return None if t is None or t.numel() == 0 else t.data_ptr()


class _Call:
    """One call's device and stream: every tensor must lie on that device."""

    def __init__(self, stream, **tensors):
        self.device = None
        for name, t in tensors.items():
            if t is None:
                continue
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            if self.device is None:
                self.device = t.device
            if t.device != self.device:
                raise ValueError(f"{name} must be on {self.device}, like the other tensors")
            if t.requires_grad and torch.is_grad_enabled():
                raise ValueError(f"{name} requires grad: this call records no graph (use torch.no_grad())")
        if stream is not None and stream.device != self.device:
            raise ValueError(f"stream must belong to {self.device}")
        self.stream = torch.cuda.current_stream(self.device) if stream is None else stream
        self._ctx = torch.cuda.stream(self.stream)   # also makes its device the current one

    def __enter__(self):
        self._ctx.__enter__()
        return ctypes.c_void_p(self.stream.cuda_stream)

    def __exit__(self, *a):
        return self._ctx.__exit__(*a)


def _heads(t, name):
    """A [heads, tokens, d] or [batch, heads, tokens, d] tensor as 4-D."""
    if t.dim() == 3:
        t = t.unsqueeze(0)
    if t.dim() != 4:
        raise ValueError(f"{name} must be [heads, tokens, d] or [batch, heads, tokens, d]")
    if t.shape[3] > 1 and t.stride(3) != 1:
        raise ValueError(f"the channels of {name} must be contiguous")
    return t


def _view(t):
    return httm_view(_data(t), t.stride(0), t.stride(1), t.stride(2))


def _same(t, like, name, dtype=None):
    if tuple(t.shape) != tuple(like.shape) or t.dtype != (dtype or like.dtype):
        raise ValueError(f"{name} must be {dtype or like.dtype} {list(like.shape)}")


def _workspace(workspace, need, device):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.device != device:
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
    return workspace


# ------------------------------------------------------------------ attention
def _attention(q, k, v, key_begin, key_end, softmax_scale):
    q, k, v = _heads(q, "q"), _heads(k, "k"), _heads(v, "v")
    B, H, L, d = q.shape
    K, N = k.shape[1], k.shape[2]
    if k.shape[0] != B or k.shape[3] != d or tuple(v.shape) != tuple(k.shape):
        raise ValueError("k and v must be [batch, kv_heads, kv_len, d] with q's batch and d")
    if q.dtype not in _DTYPES or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k and v must have one type, bfloat16 (float32 is not supported by the kernels)")
    for name, t in (("key_begin", key_begin), ("key_end", key_end)):
        if t is not None and (t.dtype != torch.int32 or tuple(t.shape) not in ((B, L), (L,) if B == 1 else (B, L))
                              or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous int32 [{B}, {L}] tensor")
    cfg = httm_attention(B, H, K, L, N, d, _DTYPES[q.dtype], float(softmax_scale), _data(key_begin), _data(key_end))
    return cfg, q, k, v


def httm_attention_workspace_bytes(batch, heads, kv_heads, q_len, kv_len, d_head, dtype=torch.bfloat16):
    """(forward, backward) workspace bytes; no device call."""
    cfg = httm_attention(batch, heads, kv_heads, q_len, kv_len, d_head, _DTYPES[dtype], 0.0, None, None)
    return _attention_bytes(cfg)


def _attention_bytes(cfg):
    f, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(load_library().httm_attention_workspace_bytes(_ref(cfg), _ref(f), _ref(b)),
           "httm_attention_workspace_bytes")
    return f.value, b.value


def httm_attention_forward(q, k, v, key_begin=None, key_end=None, softmax_scale=0.0, out=None, lse=None,
                           workspace=None, stream=None):
    """Attention of each query over its keys [key_begin, key_end).

    q: [batch, heads, q_len, d] bfloat16 (or [heads, q_len, d]), k and v:
    [batch, kv_heads, kv_len, d]; any strides with contiguous channels.
    key_begin, key_end: int32 [batch, q_len] or None (0 / kv_len); see
    :func:`causal_ranges`, :func:`frame_ranges`, :func:`length_ranges`.
    softmax_scale 0 is 1 / sqrt(d).  Returns (out like q, lse float32
    [batch, heads, q_len])."""
    call = _Call(stream, q=q, k=k, v=v, key_begin=key_begin, key_end=key_end, out=out, lse=lse, workspace=workspace)
    with call as s:
        cfg, q4, k4, v4 = _attention(q, k, v, key_begin, key_end, softmax_scale)
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        _same(out, q, "out")
        if lse is None:
            lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
        _same(lse, q[..., 0], "lse", torch.float32)
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")
        ws = _workspace(workspace, _attention_bytes(cfg)[0], call.device)
        vq, vk, vv, vo = _view(q4), _view(k4), _view(v4), _view(_heads(out, "out"))
        _check(load_library().httm_attention_forward(_ref(cfg), _ref(vq), _ref(vk), _ref(vv), _ref(vo), _data(lse),
                                                     _data(ws), ws.numel(), s), "httm_attention_forward")
    return out, lse


def httm_attention_backward(dout, q, k, v, out, lse, key_begin=None, key_end=None, softmax_scale=0.0, dq=None,
                            dk=None, dv=None, workspace=None, stream=None):
    """The gradients (dq, dk, dv) of ``sum(dout * out)`` for the q, k, v,
    ranges and scale of a :func:`httm_attention_forward` call that returned
    (out, lse).  dk and dv add up the query heads that share a key head."""
    call = _Call(stream, dout=dout, q=q, k=k, v=v, out=out, lse=lse, key_begin=key_begin, key_end=key_end, dq=dq,
                 dk=dk, dv=dv, workspace=workspace)
    with call as s:
        cfg, q4, k4, v4 = _attention(q, k, v, key_begin, key_end, softmax_scale)
        _same(dout, q, "dout")
        _same(out, q, "out")
        _same(lse, q[..., 0], "lse", torch.float32)
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")
        dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=t.device) if g is None else g
                      for g, t in ((dq, q), (dk, k), (dv, v)))
        for name, g, t in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
            _same(g, t, name)
        ws = _workspace(workspace, _attention_bytes(cfg)[1], call.device)
        views = [_view(_heads(t, n)) for t, n in ((dout, "dout"), (q4, "q"), (k4, "k"), (v4, "v"), (out, "out"))]
        grads = [_view(_heads(t, n)) for t, n in ((dq, "dq"), (dk, "dk"), (dv, "dv"))]
        _check(load_library().httm_attention_backward(_ref(cfg), *map(_ref, views), _data(lse), *map(_ref, grads),
                                                      _data(ws), ws.numel(), s), "httm_attention_backward")
    return dq, dk, dv


def causal_ranges(batch, q_len, kv_len, window=None, device="cuda"):
    """(key_begin, key_end) of causal attention: the queries are the last
    q_len tokens of the keys, each sees itself and what came before (with
    ``window``: the last `window` of those)."""
    end = torch.arange(1, q_len + 1, device=device) + (kv_len - q_len)
    begin = torch.zeros_like(end) if window is None else end - window
    return tuple(t.clamp(0, kv_len).int().expand(batch, q_len).contiguous() for t in (begin, end))


def frame_ranges(batch, q_len, kv_len, frame, device="cuda"):
    """(key_begin, key_end) of frame-causal attention: every token sees its
    whole frame of `frame` tokens and the frames before it."""
    at = torch.arange(q_len, device=device) + (kv_len - q_len)
    end = ((torch.div(at, frame, rounding_mode="floor") + 1) * frame).clamp(0, kv_len)
    end = end.int().expand(batch, q_len).contiguous()
    return torch.zeros_like(end), end


def length_ranges(lengths, q_len):
    """(key_begin, key_end) of a padded batch: every query of entry b sees
    the first lengths[b] keys (lengths: int tensor [batch])."""
    end = lengths.int()[:, None].expand(lengths.numel(), q_len).contiguous()
    return torch.zeros_like(end), end


# ------------------------------------------------------------------ rotary
def rotary_frequencies(pairs, base=10000.0, scaling=None, scale=1.0, original_length=4096, fast=32.0, slow=1.0,
                       device="cuda"):
    """(float64 radians per position of each pair, factor on cosine and
    sine).  ``scaling`` stretches them for sequences `scale` times as long as
    the trained ones: None; "linear" (positions interpolated); "ntk" (the
    base raised so that the slowest pair is interpolated and the fastest
    kept); "yarn" (pairs of under `slow` turns in `original_length`
    positions interpolated, those of over `fast` kept, a ramp between, and
    factor 0.1 ln(scale) + 1)."""
    n = torch.arange(pairs, dtype=torch.float64)
    if scaling == "ntk" and pairs > 1:
        base = base * scale ** (pairs / (pairs - 1))
    f = base ** (-n / pairs)
    factor = 1.0
    if scaling == "linear":
        f = f / scale
    elif scaling == "yarn":
        turns = original_length * f / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0, 1)
        f = f * keep + f / scale * (1 - keep)
        factor = 0.1 * math.log(scale) + 1.0 if scale > 1 else 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'yarn'")
    return f.to(device), factor


def httm_rotary(q, k, freqs, positions, axes=1, layout=HTTM_ROTARY_HALF, factor=1.0, inverse=False, q_out=None,
                k_out=None, stream=None):
    """Turns the first 2 * axes * len(freqs) channels of every head by its
    token's positions (``inverse``: back, which maps gradients).

    q: [batch, heads, tokens, d] bfloat16 or float32 (or [heads, tokens, d]),
    k: the same with its own heads, or None; any strides with contiguous
    channels, so views of a packed projection work.  positions: contiguous
    int32 [batch, tokens, axes], or [tokens, axes] / (axes 1) [tokens]
    shared by the batch.  Outputs default to new contiguous tensors in the
    [batch, heads, tokens, d] order; q_out=q turns in place.  Returns (q_out,
    k_out)."""
    call = _Call(stream, q=q, k=k, freqs=freqs, positions=positions, q_out=q_out, k_out=k_out)
    with call as s:
        q4 = _heads(q, "q")
        B, H, T, d = q4.shape
        if q.dtype not in _DTYPES:
            raise ValueError("q must be bfloat16 or float32")
        k4 = None if k is None else _heads(k, "k")
        if k4 is not None and (k4.shape[0] != B or k4.shape[2] != T or k4.shape[3] != d or k.dtype != q.dtype):
            raise ValueError("k must have q's batch, tokens, channels and type")
        if freqs.dtype != torch.float64 or freqs.dim() != 1 or not freqs.is_contiguous():
            raise ValueError("freqs must be a contiguous float64 [pairs] tensor")
        shapes = [(B, T, axes), (T, axes)] + ([(T,)] if axes == 1 else [])
        if positions.dtype != torch.int32 or tuple(positions.shape) not in shapes or not positions.is_contiguous():
            raise ValueError(f"positions must be a contiguous int32 [{B}, {T}, {axes}] or [{T}, {axes}] tensor")
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        _same(q_out, q, "q_out")
        if k is not None:
            if k_out is None:
                k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
            _same(k_out, k, "k_out")
        elif k_out is not None:
            raise ValueError("k_out without k")
        cfg = httm_rotary_cfg(B, T, H, 0 if k is None else k4.shape[1], d, _DTYPES[q.dtype], axes, freqs.numel(),
                              layout, int(bool(inverse)), float(factor), _data(positions),
                              T * axes if positions.dim() == 3 else 0, _data(freqs))
        views = [_view(q4), _view(_heads(q_out, "q_out"))]
        views += [None, None] if k is None else [_view(k4), _view(_heads(k_out, "k_out"))]
        _check(load_library().httm_rotary(_ref(cfg), *map(_ref, views), s), "httm_rotary")
    return q_out, k_out


# ------------------------------------------------------------------ gated norm
@dataclass(frozen=True)
class Norm:
    """A LayerNorm or RMSNorm: kind, float32 weight and bias (None: 1 / 0)."""
    kind: int
    weight: torch.Tensor | None = None
    bias: torch.Tensor | None = None
    eps: float = 1e-5


_NO_NORM = Norm(HTTM_NORM_NONE)


def _rows(t, shape, name, dtype):
    if tuple(t.shape) != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} {list(shape)}")
    if shape[1] > 1 and shape[0] > 0 and t.stride(1) != 1:
        raise ValueError(f"the channels of {name} must be contiguous")
    return httm_rows(_data(t), t.stride(0) if shape[0] > 1 else shape[1])


def _norm_cfg(rows, channels, stream_dtype, branch_dtype, gate, post, pre, residual_scale):
    for name, dt in (("stream", stream_dtype), ("branch", branch_dtype)):
        if dt not in _DTYPES:
            raise ValueError(f"the {name} must be bfloat16 or float32")
    post, pre = post or _NO_NORM, pre or _NO_NORM
    gates = 0
    if gate is not None:
        if gate.dim() == 1:
            gate = gate.unsqueeze(0)
        gates = gate.shape[0]
        if gate.dim() != 2 or gate.shape[1] != channels or gates == 0:
            raise ValueError(f"gate must be [{channels}] or [gates, {channels}]")
    params = dict(zip(_PARAMS, (gate, post.weight, post.bias, pre.weight, pre.bias)))
    for name, t in params.items():
        if t is None:
            continue
        if t.dtype != torch.float32 or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous float32")
        if name != "gate" and tuple(t.shape) != (channels,):
            raise ValueError(f"{name} must be [{channels}]")
    cfg = httm_norm_cfg(rows, channels, _DTYPES[stream_dtype], _DTYPES[branch_dtype], post.kind, pre.kind, gates,
                        post.eps, pre.eps, float(residual_scale))
    return cfg, params, httm_norm_weights(*(_data(t) for t in params.values()))


def _norm_tensors(gate, post, pre):
    out = dict(gate=gate)
    for side, n in (("post", post), ("pre", pre)):
        if n is not None:
            out[side + "_weight"], out[side + "_bias"] = n.weight, n.bias
    return out


def httm_gated_norm_forward(x, f=None, gate=None, post=None, pre=None, residual_scale=1.0, y=None, z=None, stats=None,
                            branch_dtype=None, stream=None):
    """y = residual_scale * x + gate * post(f); z = pre(y).

    x: [rows, channels], the token stream; f: the block's output, or None
    (then y is x if residual_scale is 1: the norm before a first block).
    gate: float32 [channels] or [gates, channels] (each serves rows / gates
    consecutive rows), or None.  post, pre: :class:`Norm` or None (no z).
    z has f's type (without f: ``branch_dtype``, or x's).  y=x updates the
    stream in place.  Returns (y, z or None, stats float32 [4, rows] for the
    backward call)."""
    call = _Call(stream, x=x, f=f, y=y, z=z, stats=stats, **_norm_tensors(gate, post, pre))
    with call as s:
        if x.dim() != 2:
            raise ValueError("x must be [rows, channels]")
        shape = tuple(x.shape)
        bdt = f.dtype if f is not None else branch_dtype or x.dtype
        cfg, _, w = _norm_cfg(*shape, x.dtype, bdt, gate, post, pre, residual_scale)
        keep_x = f is None and y is None and residual_scale == 1.0 and pre is not None
        if y is None and not keep_x:
            y = torch.empty(shape, dtype=x.dtype, device=x.device)
        if pre is None and z is not None:
            raise ValueError("z without pre")
        if pre is not None and z is None:
            z = torch.empty(shape, dtype=bdt, device=x.device)
        if stats is None:
            stats = torch.empty((4, shape[0]), dtype=torch.float32, device=x.device)
        if stats.dtype != torch.float32 or tuple(stats.shape) != (4, shape[0]) or not stats.is_contiguous():
            raise ValueError(f"stats must be a contiguous float32 [4, {shape[0]}] tensor")
        rx = _rows(x, shape, "x", x.dtype)
        rf = None if f is None else _rows(f, shape, "f", bdt)
        ry = None if y is None else _rows(y, shape, "y", x.dtype)
        rz = None if z is None else _rows(z, shape, "z", bdt)
        _check(load_library().httm_gated_norm_forward(_ref(cfg), _ref(w), _ref(rx), _ref(rf), _ref(ry), _ref(rz),
                                                      _data(stats), s), "httm_gated_norm_forward")
    return (x if keep_x else y), z, stats


def httm_gated_norm_backward(dy, dz, f, y, stats, gate=None, post=None, pre=None, residual_scale=1.0, dx=None, df=None,
                             workspace=None, stream=None):
    """The gradients of ``sum(dy * y) + sum(dz * z)`` of a
    :func:`httm_gated_norm_forward` call with the same f, gate, norms and
    scale that returned (y, z, stats).  dy may be None (0).  Returns a dict:
    dx, df, dgate, dpost_weight, dpost_bias, dpre_weight, dpre_bias; None
    where the forward call had no such input."""
    call = _Call(stream, dy=dy, dz=dz, f=f, y=y, stats=stats, dx=dx, df=df, workspace=workspace,
                 **_norm_tensors(gate, post, pre))
    with call as s:
        if y.dim() != 2:
            raise ValueError("y must be [rows, channels]")
        if (dz is None) != (pre is None):
            raise ValueError("dz must be given exactly when pre is")
        shape = tuple(y.shape)
        bdt = f.dtype if f is not None else dz.dtype if dz is not None else y.dtype
        cfg, params, w = _norm_cfg(*shape, y.dtype, bdt, gate, post, pre, residual_scale)
        if stats.dtype != torch.float32 or tuple(stats.shape) != (4, shape[0]) or not stats.is_contiguous():
            raise ValueError(f"stats must be a contiguous float32 [4, {shape[0]}] tensor")
        if dx is None:
            dx = torch.empty(shape, dtype=y.dtype, device=y.device)
        if f is None and df is not None:
            raise ValueError("df without f")
        if f is not None and df is None:
            df = torch.empty(shape, dtype=bdt, device=y.device)
        grads = {n: None if t is None else torch.empty_like(t) for n, t in params.items()}
        g = httm_norm_grads(*(_data(t) for t in grads.values()))
        need = ctypes.c_size_t(0)
        _check(load_library().httm_gated_norm_workspace_bytes(_ref(cfg), _ref(need)), "httm_gated_norm_workspace_bytes")
        ws = _workspace(workspace, need.value if any(t is not None for t in grads.values()) else 0, call.device)
        sdt = y.dtype
        rows = [None if t is None else _rows(t, shape, n, dt) for t, n, dt in
                ((dy, "dy", sdt), (dz, "dz", bdt), (f, "f", bdt), (y, "y", sdt))]
        outs = [None if t is None else _rows(t, shape, n, dt) for t, n, dt in ((dx, "dx", sdt), (df, "df", bdt))]
        _check(load_library().httm_gated_norm_backward(_ref(cfg), _ref(w), *map(_ref, rows), _data(stats),
                                                       *map(_ref, outs), _ref(g), _data(ws), ws.numel(), s),
               "httm_gated_norm_backward")
        if gate is not None and gate.dim() == 1:
            grads["gate"] = grads["gate"][0]
    return dict(dx=dx, df=df, **{"d" + n: t for n, t in grads.items()})


def httm_ops_device_status(device=None, stream=None) -> int:
    """Synchronises the stream; returns the HTTM_DEV_* bits the operators'
    kernels set on the device since the last call (0 = clean)."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    v = ctypes.c_uint32(0)
    with torch.cuda.device(device):
        s = torch.cuda.current_stream(device) if stream is None else stream
        st = load_library().httm_ops_device_status(ctypes.c_void_p(s.cuda_stream), ctypes.byref(v))
    if st not in (0, 7, 8):
        _check(st, "httm_ops_device_status")
    return int(v.value)
