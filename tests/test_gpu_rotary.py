"""Rotary positions against their definition in 64 bits."""
from __future__ import annotations

import pytest
import torch

import oplib
from token_merging_view_b200 import ops

pytestmark = pytest.mark.gpu

HALF, PAIRS = ops.HTTM_ROTARY_HALF, ops.HTTM_ROTARY_PAIRS


def _rand(shape, seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _check(x, got, freqs, pos, axes, layout, factor, inverse, name):
    pos = pos.view(-1, x.shape[2], axes)
    want = oplib.rotary(x, freqs, pos, axes, layout == HALF, factor, inverse)
    e, u = oplib.rotary_tol(x, freqs, pos, axes, layout == HALF, factor, x.dtype)
    # fp32 sums of two rounded products: 3 roundings of their magnitudes, within e's 2^-21
    oplib.check(got, want, e + u * (want.abs() + e), name)
    rot = 2 * axes * freqs.numel()
    assert torch.equal(got[..., rot:], x[..., rot:]), "channels behind the turned ones are copied"


CASES = [
    # B, T, H, K, d, axes, pairs, layout, dtype, far
    (1, 1, 1, 0, 2, 1, 1, HALF, torch.float32, 0),
    (2, 37, 4, 2, 64, 2, 16, HALF, torch.bfloat16, 0),
    (2, 37, 4, 2, 64, 1, 32, HALF, torch.bfloat16, 1 << 20),
    (1, 100, 3, 1, 64, 1, 16, PAIRS, torch.bfloat16, 1 << 20),
    (1, 100, 3, 1, 64, 1, 8, HALF, torch.float32, 1 << 20),
    (3, 5, 2, 2, 50, 1, 13, HALF, torch.float32, 1 << 30),
    (3, 5, 2, 2, 51, 2, 9, PAIRS, torch.bfloat16, 100),
    (1, 2000, 1, 1, 128, 4, 16, HALF, torch.bfloat16, 500),
    (1, 9, 5, 3, 40, 3, 4, PAIRS, torch.float32, 500),
    (16, 1, 32, 8, 128, 1, 64, PAIRS, torch.bfloat16, 1 << 24),
    (2, 3, 1, 1, 24, 1, 4, HALF, torch.bfloat16, 9),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("inverse", [False, True])
def test_against_definition(case, inverse):
    B, T, H, K, d, axes, pairs, layout, dtype, far = case
    q = _rand((B, H, T, d), 1, dtype)
    k = _rand((B, K, T, d), 2, dtype) if K else None
    g = torch.Generator(device="cuda").manual_seed(3)
    pos = torch.randint(-far, far + 1, (B, T, axes), generator=g, device="cuda").int()
    freqs, factor = ops.rotary_frequencies(pairs, base=500.0, scaling="yarn", scale=3.0)
    qo, ko = ops.httm_rotary(q, k, freqs, pos, axes=axes, layout=layout, factor=factor, inverse=inverse)
    _check(q, qo, freqs, pos, axes, layout, factor, inverse, "q")
    if K:
        _check(k, ko, freqs, pos, axes, layout, factor, inverse, "k")
    assert ops.httm_ops_device_status() == 0


def test_any_frequency():
    """Negative, zero, above a turn per position."""
    q = _rand((1, 2, 300, 16), 1, torch.float32)
    freqs = torch.tensor([0.0, -1.0, 100.5, 6.283185307179586, -7e-9, 1e-300, 3.0, -0.25], dtype=torch.float64, device="cuda")
    pos = torch.arange(-150, 150, device="cuda").int()
    out, _ = ops.httm_rotary(q, None, freqs, pos)
    _check(q, out, freqs, pos, 1, HALF, 1.0, False, "q")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", [HALF, PAIRS])
def test_layouts_strides_and_in_place(dtype, layout):
    """A packed projection into [heads, tokens, d], odd strides and bases,
    shared positions, and in place: the same bits."""
    B, T, H, d = 2, 65, 3, 64
    packed = _rand((B, T, 3, H, d), 4, dtype)
    q, k = packed[:, :, 0].transpose(1, 2), packed[:, :, 1].transpose(1, 2)
    freqs, _ = ops.rotary_frequencies(32)
    pos = torch.arange(T, device="cuda").int()
    kw = dict(freqs=freqs, positions=pos, layout=layout)
    qo, ko = ops.httm_rotary(q, k, **kw)
    assert qo.is_contiguous()
    both = pos[:, None].expand(B, T, 1).contiguous()
    q2, k2 = ops.httm_rotary(q.contiguous(), k.contiguous(), freqs, both, layout=layout)
    assert torch.equal(qo, q2) and torch.equal(ko, k2)
    odd = torch.zeros((B, H, T, d + 3), dtype=dtype, device="cuda")     # rows that start off 16 bytes
    q3, _ = ops.httm_rotary(q, None, q_out=odd[..., 1:d + 1], **kw)
    assert torch.equal(q3, qo) and (odd[..., 0] == 0).all() and (odd[..., d + 1:] == 0).all()
    q4, _ = ops.httm_rotary(odd[..., 1:d + 1], None, inverse=True, **kw)
    q5, _ = ops.httm_rotary(qo, None, inverse=True, **kw)
    assert torch.equal(q4, q5)
    v = packed[:, :, 2].clone()
    ops.httm_rotary(q, k, q_out=q, k_out=k, **kw)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(packed[:, :, 2], v)


def test_back_and_forth_and_gradient():
    """The inverse turn undoes the turn (fp32), and is the gradient: <turn(x),
    g> = <x, inverse(g)>."""
    x, g = _rand((1, 2, 50, 32), 1, torch.float32), _rand((1, 2, 50, 32), 2, torch.float32)
    freqs, _ = ops.rotary_frequencies(8, base=100.0)
    pos = torch.randint(0, 1000, (50, 2), device="cuda").int()
    y, _ = ops.httm_rotary(x, None, freqs, pos, axes=2)
    b, _ = ops.httm_rotary(g, None, freqs, pos, axes=2, inverse=True)
    z, _ = ops.httm_rotary(y, None, freqs, pos, axes=2, inverse=True)
    assert (z - x).abs().max() <= 4 * 2.0 ** -20 * x.abs().max()        # two turns of 2^-21 (|a| + |b|) each
    lhs, rhs = (y.double() * g.double()).sum(), (x.double() * b.double()).sum()
    mag = 2.0 ** -20 * ((y.double().abs() + x.double().abs().amax()) * (g.double().abs() + g.double().abs().amax())).sum()
    assert (lhs - rhs).abs() <= mag


def test_no_tokens_and_graph():
    freqs, _ = ops.rotary_frequencies(32)
    e, _ = ops.httm_rotary(torch.empty((2, 3, 0, 64), device="cuda"), None, freqs,
                           torch.empty((0,), dtype=torch.int32, device="cuda"))
    assert e.shape == (2, 3, 0, 64)
    x, pos = _rand((1, 2, 7, 64), 1, torch.bfloat16), torch.arange(7, device="cuda").int()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y, _ = ops.httm_rotary(x, None, freqs, pos)
    x.mul_(-2)
    pos.add_(1000)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, ops.httm_rotary(x, None, freqs, pos)[0])


def test_refusals():
    x = torch.zeros((2, 4, 8, 64), device="cuda")
    freqs, _ = ops.rotary_frequencies(32)
    pos = torch.zeros(8, dtype=torch.int32, device="cuda")
    for bad in (dict(q=x.half()), dict(q=x.transpose(2, 3)), dict(q=x[0, 0]), dict(k=x.bfloat16()), dict(k=x[:, :, :4]),
                dict(freqs=freqs.float()), dict(positions=pos.long()), dict(positions=pos[:7]), dict(axes=2),
                dict(q_out=x.bfloat16()), dict(q_out=x[:1]), dict(freqs=freqs.cpu()), dict(k_out=x)):
        with pytest.raises((ValueError, ops.HttmError)):
            ops.httm_rotary(**{**dict(q=x, k=None, freqs=freqs, positions=pos), **bad})
    with pytest.raises(ops.HttmError):
        ops.httm_rotary(x, None, torch.ones(33, dtype=torch.float64, device="cuda"), pos)    # 66 channels of 64
    with pytest.raises(ops.HttmError):
        ops.httm_rotary(x, None, freqs, pos, q_out=torch.zeros((2, 1, 8, 64), device="cuda").expand(2, 4, 8, 64))
    with pytest.raises(ValueError, match="requires grad"):
        ops.httm_rotary(x.clone().requires_grad_(), None, freqs, pos)


@pytest.mark.parametrize("sign", [1, -1])
def test_angles_are_as_good_near_quarter_turns_as_near_zero(sign):
    """(1, 0) turned is (cos, sin): each within 6 roundings of itself (the
    angle behind the nearest quarter turn is rounded once, and moves sine or
    cosine by less than that relative to the value; 4 are the function's, at
    most 2 steps; 1 the result's) and what 64 bits lose of position *
    frequency, 2^-50 of it."""
    pairs, T = 4, 200000
    freqs = torch.tensor([1.0, 0.37, 2.0 ** -9 * 3.141592653589793, 1e-5], dtype=torch.float64, device="cuda")
    x = torch.zeros((1, 1, T, 2 * pairs), device="cuda")
    x[..., :pairs] = 1.0
    pos = (sign * torch.arange(T, device="cuda")).int()
    out, _ = ops.httm_rotary(x, None, freqs, pos, layout=HALF)
    ang = pos.double()[:, None] * freqs
    want = torch.cat([torch.cos(ang), torch.sin(ang)], -1)
    bound = 6 * 2.0 ** -24 * want.abs() + 2.0 ** -50 * ang.abs().repeat(1, 2) + 2.0 ** -60
    assert ((out[0, 0].double() - want).abs() <= bound).all()
