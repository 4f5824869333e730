"""The operators run together, as one attention block: forward and gradients
against the block in 64 bits, the merged layer behind the same front end, and
a step captured into a graph."""
from __future__ import annotations

import math

import pytest
import torch

import oplib
from token_merging_view_b200 import GlobalAttentionBlock, Norm, grid_positions, ops
from token_merging_view_b200 import binding as B

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
H, D, C, T, GRID = 4, 64, 256, 3, 13
N = T * GRID * GRID


def _rand(shape, seed, dtype=torch.float32, scale=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale + mean).to(dtype)


def _orthogonal(rows, cols, seed):
    """Rows or columns orthonormal: the map neither stretches nor shrinks an error."""
    blocks = [torch.linalg.qr(_rand((cols, cols), seed + i))[0] for i in range(rows // cols)]
    return torch.cat(blocks).to(BF)


def _block():
    norm = lambda s: Norm(ops.HTTM_NORM_LAYER, _rand((C,), s, scale=0.1, mean=1.0), _rand((C,), s + 1, scale=0.1))  # noqa: E731
    freqs, _ = ops.rotary_frequencies(D // 4, base=100.0)
    return GlobalAttentionBlock(heads=H, qkv_weight=_orthogonal(3 * C, C, 1), proj_weight=_orthogonal(C, C, 9),
                                gate=_rand((C,), 11, scale=0.2, mean=1.0), norm1=norm(12), norm2=norm(14), freqs=freqs)


def _exact(block, x, pos, begin, end):
    """(y, z', leaves) of the block in 64 bits, with autograd."""
    leaves = {k: t.double().requires_grad_() for k, t in dict(
        dx=x, dqkv_weight=block.qkv_weight, dproj_weight=block.proj_weight, dgate=block.gate,
        dnorm1_weight=block.norm1.weight, dnorm1_bias=block.norm1.bias, dnorm2_weight=block.norm2.weight,
        dnorm2_bias=block.norm2.bias).items()}
    ln = lambda v, w, b: torch.nn.functional.layer_norm(v, (C,), w, b, 1e-5)  # noqa: E731
    z = ln(leaves["dx"], leaves["dnorm1_weight"], leaves["dnorm1_bias"])
    q, k, v = (z @ leaves["dqkv_weight"].t()).view(N, 3, H, D).permute(1, 2, 0, 3)
    ang = (pos.double()[:, :, None] * block.freqs).view(N, 2, 1, D // 4)            # [N, axis, 1, pairs]
    rot = torch.polar(torch.ones_like(ang), ang)
    turn = lambda t: torch.view_as_real(torch.complex(*t.view(H, N, 2, 2, D // 4).unbind(3)) * rot[:, :, 0]).transpose(-1, -2).reshape(H, N, D)  # noqa: E731
    s = turn(q) @ turn(k).transpose(1, 2) / math.sqrt(D)
    j = torch.arange(N, device="cuda")
    if begin is not None:
        s = s.masked_fill((j < begin[:, None]) | (j >= end[:, None]), -math.inf)
    o = torch.softmax(s, -1) @ v
    y = leaves["dx"] + leaves["dgate"] * (o.transpose(0, 1).reshape(N, C) @ leaves["dproj_weight"].t())
    return y, ln(y, leaves["dnorm2_weight"], leaves["dnorm2_bias"]), leaves


@pytest.mark.parametrize("frames", [False, True])
def test_block_against_64_bits(frames):
    """A rounding to bf16 moves a tensor by at most U of its 2-norm.  From x
    to z' and back to any gradient the block rounds fewer than 24 times (z,
    packed heads, q, k, P, o, f, y, z', df, do, P, dS, dq, dk, dv, dz, dx and
    the matrix products' results); the maps between are orthogonal, averages
    or norms of unit gain, so each output is within 24 U of its norm."""
    block, pos = _block(), grid_positions(T, GRID)
    x, dy, dz = _rand((N, C), 20, BF), _rand((N, C), 21, BF), _rand((N, C), 22, BF)
    b, e = (t[0] for t in ops.frame_ranges(1, N, N, GRID * GRID)) if frames else (None, None)
    y, z, saved = block.forward(x, pos, key_begin=b, key_end=e)
    grads = block.backward(dy, dz, saved)
    assert ops.httm_ops_device_status() == 0
    y64, z64, leaves = _exact(block, x, pos, b, e)
    want = torch.autograd.grad((y64 * dy.double()).sum() + (z64 * dz.double()).sum(), list(leaves.values()))
    for name, got, ref in [("y", y, y64.detach()), ("z", z, z64.detach())] + \
            [(k, grads[k], w) for k, w in zip(leaves, want)]:
        err = float((got.double() - ref).norm() / ref.norm())
        assert err <= 24 * oplib.U, (name, err)


def test_handing_z_from_block_to_block():
    """norm2 of one block is norm1 of the next: the same y as letting the
    second block norm the stream itself, and the same gradients."""
    first, second, pos = _block(), _block(), grid_positions(T, GRID)
    second.norm1 = first.norm2
    x, dy, dz = _rand((N, C), 20, BF), _rand((N, C), 21, BF), _rand((N, C), 22, BF)
    y1, z1, _ = first.forward(x, pos)
    y2, z2, s2 = second.forward(y1, pos, z=z1)
    y3, z3, s3 = second.forward(y1, pos)
    assert torch.equal(y2, y3) and torch.equal(z2, z3)
    g2, g3 = second.backward(dy, dz, s2), second.backward(dy, dz, s3)
    assert torch.equal(g2["dqkv_weight"], g3["dqkv_weight"]) and torch.equal(g2["dgate"], g3["dgate"])
    assert g3["dnorm1_weight"] is not None and g2["dnorm1_weight"] is None and "dz" in g2


def test_merged_layer_behind_the_same_front_end():
    """With a plan that merges nothing the merged layer is dense attention
    over the same q, k, v; with one that merges, it runs and differs."""
    block, pos = _block(), grid_positions(T, GRID)
    x = _rand((N, C), 20, BF)
    y, z, saved = block.forward(x, pos)
    cfg = dict(h=H, T=T, P=GRID * GRID, d_head=D, n_s=32, n_t=3)
    none = B.httm_plan(B.LayerConfig(**cfg, q_merge_pct=0, kv_merge_pct=0, outlier_pct=0))
    ym, zm, nothing = block.forward(x, pos, plan=none)
    assert nothing is None
    # o, f and y are rounded apart in the two paths: three roundings of each side
    assert float((ym.double() - y.double()).norm() / y.double().norm()) <= 6 * oplib.U
    some = B.httm_plan(B.LayerConfig(**cfg, q_merge_pct=50, kv_merge_pct=50, outlier_pct=10))
    ys, _, _ = block.forward(x, pos, plan=some)
    assert torch.isfinite(ys).all() and not torch.equal(ys, y)
    with pytest.raises(ValueError, match="no gradient"):
        block.backward(x, x, nothing)
    with pytest.raises(ValueError, match="key ranges"):
        block.forward(x, pos, plan=none, key_end=torch.full((N,), N, dtype=torch.int32, device="cuda"))


def test_training_step_in_a_graph():
    block, pos = _block(), grid_positions(T, GRID)
    x, dy, dz = _rand((N, C), 20, BF), _rand((N, C), 21, BF), _rand((N, C), 22, BF)

    def step():
        y, z, saved = block.forward(x, pos)
        return dict(block.backward(dy, dz, saved), y=y, z=z)

    step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    for t in (x, dy, dz):
        t.copy_(t.flip(0))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    want = step()
    for n, t in want.items():
        assert torch.equal(got[n], t), n
