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
from struct import Struct

import torch

from .binding import HTTM_BF16, HTTM_F32, HttmError, _check, load_library  # noqa: F401

HTTM_ROTARY_HALF, HTTM_ROTARY_PAIRS = 0, 1
HTTM_NORM_NONE, HTTM_NORM_LAYER, HTTM_NORM_RMS = 0, 1, 2

_DTYPES = {torch.bfloat16: HTTM_BF16, torch.float32: HTTM_F32}
_PARAMS = ("gate", "post_weight", "post_bias", "pre_weight", "pre_bias")

# The C structs of include/httm.h as byte strings: small calls are bound by
# the host, and packing one is several times cheaper than a ctypes.Structure.
# Pointers are passed as integers (0: NULL); "0q" pads to a multiple of 8.
httm_view = Struct("@P3q").pack             # data, batch, head, token strides
httm_attention = Struct("@7if2P").pack      # batch .. dtype, softmax_scale, key_begin, key_end
httm_rotary_cfg = Struct("@10ifPqP").pack   # batch .. inverse, factor, positions, position_batch, freqs
httm_norm_cfg = Struct("@q6i3f0q").pack     # rows, channels .. gates, post_eps, pre_eps, residual_scale
httm_rows = Struct("@Pq").pack              # data, row stride
httm_norm_weights = httm_norm_grads = Struct("@5P").pack   # in the order of _PARAMS

# The current device and raw stream, the short way where this torch has one (a
# torch without CUDA has not, and can still import the package and plan).
_device_of_thread = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _data(t):
    return 0 if t is None else t.data_ptr()


def _common_device(named):
    """The index of the one device all these tensors lie on."""
    device, first = -1, None
    grad = torch.is_grad_enabled()
    for name, t in named:
        if t is None:
            continue
        i = t.get_device() if isinstance(t, torch.Tensor) else -1
        if i < 0:
            raise ValueError(f"{name} must be a CUDA tensor")
        if device < 0:
            device, first = i, name
        elif i != device:
            raise ValueError(f"{name} must be on the device of {first}, cuda:{device}")
        if grad and t.requires_grad:
            raise ValueError(f"{name} requires grad: this call records no graph (use torch.no_grad())")
    return device


class _On:
    """Makes the tensors' device (and `stream`, if given) the current one for
    one call; yields the raw stream.  Costs nothing where both are already."""
    __slots__ = ("device", "stream", "ctx")

    def __init__(self, device, stream):
        self.device, self.stream = device, stream

    def __enter__(self):
        self.ctx = None
        if self.stream is None and _device_of_thread() == self.device:
            return _raw_stream(self.device)
        stream = self.stream
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        elif stream.device.index != self.device:
            raise ValueError(f"stream must belong to cuda:{self.device}")
        self.ctx = torch.cuda.stream(stream)         # its device too
        self.ctx.__enter__()
        return stream.cuda_stream

    def __exit__(self, *a):
        if self.ctx is not None:
            self.ctx.__exit__(*a)


def _view(t, name):
    """The httm_view of a [heads, tokens, d] or [batch, heads, tokens, d] tensor."""
    st = t.stride()
    if len(st) == 3:
        st = (0, *st)
    elif len(st) != 4:
        raise ValueError(f"{name} must be [heads, tokens, d] or [batch, heads, tokens, d]")
    if st[3] != 1 and t.shape[-1] > 1:
        raise ValueError(f"the channels of {name} must be contiguous")
    return httm_view(t.data_ptr(), st[0], st[1], st[2])


def _heads_shape(t, name):
    s = t.shape
    if len(s) == 4:
        return s
    if len(s) == 3:
        return (1, *s)
    raise ValueError(f"{name} must be [heads, tokens, d] or [batch, heads, tokens, d]")


def _new_like(t):
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(*t.shape, dtype=t.dtype, device=t.device)


def _same(t, like, name):
    if t.shape != like.shape or t.dtype != like.dtype:
        raise ValueError(f"{name} must be {like.dtype} {list(like.shape)}")


def _workspace(workspace, need, like):
    """(pointer, bytes, the tensor to keep alive through the call)."""
    if workspace is None:
        if need == 0:
            return 0, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    return workspace.data_ptr(), workspace.numel(), workspace


# ------------------------------------------------------------------ attention
def _attention(q, k, v, key_begin, key_end, softmax_scale):
    """The httm_attention of these tensors."""
    B, H, L, d = _heads_shape(q, "q")
    ks = _heads_shape(k, "k")
    if ks[0] != B or ks[3] != d or v.shape != k.shape:
        raise ValueError("k and v must be [batch, kv_heads, kv_len, d] with q's batch and d")
    dt = q.dtype
    if dt not in _DTYPES or k.dtype != dt or v.dtype != dt:
        raise ValueError("q, k and v must have one type, bfloat16 (float32 is not supported by the kernels)")
    for name, t in (("key_begin", key_begin), ("key_end", key_end)):
        if t is not None and (t.dtype != torch.int32 or not t.is_contiguous() or
                              not (t.shape == (B, L) or (B == 1 and t.shape == (L,)))):
            raise ValueError(f"{name} must be a contiguous int32 [{B}, {L}] tensor")
    return httm_attention(B, H, ks[1], L, ks[2], d, _DTYPES[dt], softmax_scale, _data(key_begin), _data(key_end))


def httm_attention_workspace_bytes(batch, heads, kv_heads, q_len, kv_len, d_head, dtype=torch.bfloat16):
    """(forward, backward) workspace bytes of calls of these sizes, with key
    ranges or without; no device call."""
    return _attention_bytes(httm_attention(batch, heads, kv_heads, q_len, kv_len, d_head, _DTYPES[dtype], 0.0, 0, 0))


def _attention_bytes(cfg):
    n = (ctypes.c_size_t * 2)()
    st = load_library().httm_attention_workspace_bytes(cfg, ctypes.addressof(n), ctypes.addressof(n) + 8)
    if st:
        _check(st, "httm_attention_workspace_bytes")
    return n[0], n[1]


def _lse(lse, q):
    shape = q.shape[:-1]
    if lse is None:
        return torch.empty(*shape, dtype=torch.float32, device=q.device)
    if lse.shape != shape or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 {list(shape)} tensor")
    return lse


def httm_attention_forward(q, k, v, key_begin=None, key_end=None, softmax_scale=0.0, out=None, lse=None,
                           workspace=None, stream=None):
    """Attention of each query over its keys [key_begin, key_end).

    q: [batch, heads, q_len, d] bfloat16 (or [heads, q_len, d]), k and v:
    [batch, kv_heads, kv_len, d]; any strides with contiguous channels.
    key_begin, key_end: int32 [batch, q_len] or None (0 / kv_len); see
    :func:`causal_ranges`, :func:`frame_ranges`, :func:`length_ranges`.
    softmax_scale 0 is 1 / sqrt(d).  Returns (out like q, lse float32
    [batch, heads, q_len])."""
    device = _common_device((("q", q), ("k", k), ("v", v), ("key_begin", key_begin), ("key_end", key_end),
                             ("out", out), ("lse", lse), ("workspace", workspace)))
    with _On(device, stream) as s:
        cfg = _attention(q, k, v, key_begin, key_end, softmax_scale)
        if out is None:
            out = _new_like(q)
        else:
            _same(out, q, "out")
        lse = _lse(lse, q)
        ws, n, keep = _workspace(workspace, _attention_bytes(cfg)[0], q)
        st = load_library().httm_attention_forward(cfg, _view(q, "q"), _view(k, "k"), _view(v, "v"),
                                                   _view(out, "out"), lse.data_ptr(), ws, n, s)
        if st:
            _check(st, "httm_attention_forward")
    return out, lse


def httm_attention_backward(dout, q, k, v, out, lse, key_begin=None, key_end=None, softmax_scale=0.0, dq=None,
                            dk=None, dv=None, workspace=None, stream=None):
    """The gradients (dq, dk, dv) of ``sum(dout * out)`` for the q, k, v,
    ranges and scale of a :func:`httm_attention_forward` call that returned
    (out, lse).  dk and dv add up the query heads that share a key head."""
    device = _common_device((("dout", dout), ("q", q), ("k", k), ("v", v), ("out", out), ("lse", lse),
                             ("key_begin", key_begin), ("key_end", key_end), ("dq", dq), ("dk", dk), ("dv", dv),
                             ("workspace", workspace)))
    with _On(device, stream) as s:
        cfg = _attention(q, k, v, key_begin, key_end, softmax_scale)
        _same(dout, q, "dout")
        _same(out, q, "out")
        if lse is None:
            raise ValueError("lse must be the forward call's")
        lse = _lse(lse, q)
        grads = []
        for name, g, t in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
            if g is None:
                g = _new_like(t)
            else:
                _same(g, t, name)
            grads.append(g)
        dq, dk, dv = grads
        ws, n, keep = _workspace(workspace, _attention_bytes(cfg)[1], q)
        st = load_library().httm_attention_backward(
            cfg, _view(dout, "dout"), _view(q, "q"), _view(k, "k"), _view(v, "v"), _view(out, "out"), lse.data_ptr(),
            _view(dq, "dq"), _view(dk, "dk"), _view(dv, "dv"), ws, n, s)
        if st:
            _check(st, "httm_attention_backward")
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
    device = _common_device((("q", q), ("k", k), ("freqs", freqs), ("positions", positions), ("q_out", q_out),
                             ("k_out", k_out)))
    with _On(device, stream) as s:
        B, H, T, d = _heads_shape(q, "q")
        dt = q.dtype
        if dt not in _DTYPES:
            raise ValueError("q must be bfloat16 or float32")
        if freqs.dtype != torch.float64 or freqs.dim() != 1 or not freqs.is_contiguous():
            raise ValueError("freqs must be a contiguous float64 [pairs] tensor")
        ps = positions.shape
        if positions.dtype != torch.int32 or not positions.is_contiguous() or not (
                ps == (B, T, axes) or ps == (T, axes) or (axes == 1 and ps == (T,))):
            raise ValueError(f"positions must be a contiguous int32 [{B}, {T}, {axes}] or [{T}, {axes}] tensor")
        if q_out is None:
            q_out = _new_like(q)
        else:
            _same(q_out, q, "q_out")
        kv_heads, vk, vk_out = 0, None, None
        if k is not None:
            ks = _heads_shape(k, "k")
            if ks[0] != B or ks[2] != T or ks[3] != d or k.dtype != dt:
                raise ValueError("k must have q's batch, tokens, channels and type")
            if k_out is None:
                k_out = _new_like(k)
            else:
                _same(k_out, k, "k_out")
            kv_heads, vk, vk_out = ks[1], _view(k, "k"), _view(k_out, "k_out")
        elif k_out is not None:
            raise ValueError("k_out without k")
        cfg = httm_rotary_cfg(B, T, H, kv_heads, d, _DTYPES[dt], axes, freqs.shape[0], layout, 1 if inverse else 0,
                              factor, positions.data_ptr(), T * axes if len(ps) == 3 else 0, freqs.data_ptr())
        st = load_library().httm_rotary(cfg, _view(q, "q"), _view(q_out, "q_out"), vk, vk_out, s)
        if st:
            _check(st, "httm_rotary")
    return q_out, k_out


# ------------------------------------------------------------------ gated norm
@dataclass(slots=True)
class Norm:
    """A LayerNorm or RMSNorm: kind, float32 weight and bias (None: 1 / 0)."""
    kind: int
    weight: torch.Tensor | None = None
    bias: torch.Tensor | None = None
    eps: float = 1e-5


_NO_NORM = Norm(HTTM_NORM_NONE)


def _rows(t, shape, name, dtype):
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} {list(shape)}")
    row, col = t.stride()
    if col != 1 and shape[1] > 1 and shape[0] > 0:
        raise ValueError(f"the channels of {name} must be contiguous")
    return httm_rows(t.data_ptr(), row if shape[0] > 1 else shape[1])


def _norm_cfg(shape, stream_dtype, branch_dtype, gate, post, pre, residual_scale):
    """(httm_norm_cfg, httm_norm_weights, the parameters in the order of _PARAMS)."""
    if stream_dtype not in _DTYPES or branch_dtype not in _DTYPES:
        raise ValueError("the stream and the branch must be bfloat16 or float32")
    rows, channels = shape
    post, pre = post or _NO_NORM, pre or _NO_NORM
    gates = 0
    if gate is not None:
        gs = gate.shape
        gates = gs[0] if len(gs) == 2 else 1
        if gs[-1] != channels or len(gs) not in (1, 2) or gates == 0:
            raise ValueError(f"gate must be [{channels}] or [gates, {channels}]")
    params = (gate, post.weight, post.bias, pre.weight, pre.bias)
    for name, t in zip(_PARAMS, params):
        if t is None:
            continue
        if t.dtype != torch.float32 or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous float32")
        if t.shape != (channels,) and name != "gate":
            raise ValueError(f"{name} must be [{channels}]")
    cfg = httm_norm_cfg(rows, channels, _DTYPES[stream_dtype], _DTYPES[branch_dtype], post.kind, pre.kind, gates,
                        post.eps, pre.eps, residual_scale)
    return cfg, httm_norm_weights(*map(_data, params)), params


def _norm_tensors(post, pre):
    post, pre = post or _NO_NORM, pre or _NO_NORM
    return (("post_weight", post.weight), ("post_bias", post.bias), ("pre_weight", pre.weight), ("pre_bias", pre.bias))


def _stats(stats, rows, like):
    if stats is None:
        return torch.empty(4, rows, dtype=torch.float32, device=like.device)
    if stats.dtype != torch.float32 or stats.shape != (4, rows) or not stats.is_contiguous():
        raise ValueError(f"stats must be a contiguous float32 [4, {rows}] tensor")
    return stats


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
    device = _common_device((("x", x), ("f", f), ("gate", gate), ("y", y), ("z", z), ("stats", stats),
                             *_norm_tensors(post, pre)))
    with _On(device, stream) as s:
        shape, xdt = x.shape, x.dtype
        if len(shape) != 2:
            raise ValueError("x must be [rows, channels]")
        bdt = f.dtype if f is not None else branch_dtype or xdt
        cfg, weights, _ = _norm_cfg(shape, xdt, bdt, gate, post, pre, residual_scale)
        keep_x = f is None and y is None and residual_scale == 1.0 and pre is not None
        if y is None and not keep_x:
            y = _new_like(x)
        if pre is None:
            if z is not None:
                raise ValueError("z without pre")
        elif z is None:
            z = torch.empty(*shape, dtype=bdt, device=x.device)
        stats = _stats(stats, shape[0], x)
        st = load_library().httm_gated_norm_forward(
            cfg, weights, _rows(x, shape, "x", xdt), None if f is None else _rows(f, shape, "f", bdt),
            None if y is None else _rows(y, shape, "y", xdt), None if z is None else _rows(z, shape, "z", bdt),
            stats.data_ptr(), s)
        if st:
            _check(st, "httm_gated_norm_forward")
    return (x if keep_x else y), z, stats


def httm_gated_norm_backward(dy, dz, f, y, stats, gate=None, post=None, pre=None, residual_scale=1.0, dx=None, df=None,
                             workspace=None, stream=None):
    """The gradients of ``sum(dy * y) + sum(dz * z)`` of a
    :func:`httm_gated_norm_forward` call with the same f, gate, norms and
    scale that returned (y, z, stats).  dy may be None (0).  Returns a dict:
    dx, df, dgate, dpost_weight, dpost_bias, dpre_weight, dpre_bias; None
    where the forward call had no such input."""
    device = _common_device((("dy", dy), ("dz", dz), ("f", f), ("y", y), ("stats", stats), ("gate", gate), ("dx", dx),
                             ("df", df), ("workspace", workspace), *_norm_tensors(post, pre)))
    with _On(device, stream) as s:
        shape, sdt = y.shape, y.dtype
        if len(shape) != 2:
            raise ValueError("y must be [rows, channels]")
        if (dz is None) != (pre is None):
            raise ValueError("dz must be given exactly when pre is")
        if stats is None:
            raise ValueError("stats must be the forward call's")
        bdt = f.dtype if f is not None else dz.dtype if dz is not None else sdt
        cfg, weights, params = _norm_cfg(shape, sdt, bdt, gate, post, pre, residual_scale)
        stats = _stats(stats, shape[0], y)
        if dx is None:
            dx = _new_like(y)
        if f is None:
            if df is not None:
                raise ValueError("df without f")
        elif df is None:
            df = _new_like(f)
        grads = [None if t is None else torch.empty_like(t) for t in params]
        need = ctypes.c_size_t(0)
        lib = load_library()
        st = lib.httm_gated_norm_workspace_bytes(cfg, ctypes.addressof(need))
        if st:
            _check(st, "httm_gated_norm_workspace_bytes")
        ws, n, keep = _workspace(workspace, need.value if any(t is not None for t in grads) else 0, y)
        rows = [None if t is None else _rows(t, shape, name, dt) for name, t, dt in
                (("dy", dy, sdt), ("dz", dz, bdt), ("f", f, bdt), ("y", y, sdt), ("dx", dx, sdt), ("df", df, bdt))]
        st = lib.httm_gated_norm_backward(cfg, weights, *rows[:4], stats.data_ptr(), *rows[4:],
                                          httm_norm_grads(*map(_data, grads)), ws, n, s)
        if st:
            _check(st, "httm_gated_norm_backward")
    return dict(dx=dx, df=df, **{"d" + name: t for name, t in zip(_PARAMS, grads)})


def _index(device):
    index = None if device is None else torch.device(device).index
    return torch.cuda.current_device() if index is None else index   # none, or "cuda": the current one


def httm_ops_device_status(device=None, stream=None) -> int:
    """Synchronises the stream; returns the HTTM_DEV_* bits the operators'
    kernels set on the device since the last call (0 = clean)."""
    v = ctypes.c_uint32(0)
    with _On(_index(device), stream) as s:
        st = load_library().httm_ops_device_status(s, ctypes.byref(v))
    if st not in (0, 7, 8):
        _check(st, "httm_ops_device_status")
    return int(v.value)


def httm_ops_set_wait_budget(nanoseconds, device=None, stream=None) -> None:
    """Bounds every device wait of the operators on the device, from here on
    in the stream's order (2e9 to begin with; 0: whatever is not complete
    already runs out, to check the detection)."""
    if not 0 <= nanoseconds < 2 ** 64:
        raise ValueError("nanoseconds must be within 0 .. 2^64 - 1")
    with _On(_index(device), stream) as s:
        _check(load_library().httm_ops_set_wait_budget(nanoseconds, s), "httm_ops_set_wait_budget")
