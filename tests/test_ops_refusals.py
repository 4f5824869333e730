"""What the operators around the layer refuse, on the host: every case
returns its status before any device call (the pointers are not memory), and
the Python functions refuse tensors before any pointer leaves them."""
from __future__ import annotations

import ctypes
import os
import subprocess
import sys

import pytest
import torch

from token_merging_view_b200 import binding as B
from token_merging_view_b200 import ops

FAKE = 1 << 20
ARG, UNSUPPORTED, WORKSPACE, ALIGN = 1, 2, 4, 5
R = ctypes.byref


def _cfg(**kw):
    a = dict(batch=2, heads=4, kv_heads=2, q_len=100, kv_len=300, d_head=64, dtype=0, softmax_scale=0.0,
             key_begin=0, key_end=0)
    a.update(kw)
    return ops.httm_attention(*a.values())


def _view(heads, tokens, d=64, data=FAKE, **kw):
    v = dict(batch=heads * tokens * d, head=tokens * d, token=d)
    v.update(kw)
    return ops.httm_view(data, v["batch"], v["head"], v["token"])


def _forward(cfg=None, q=None, k=None, v=None, out=None, lse=FAKE, ws=FAKE, n=0, **kw):
    cfg = cfg or _cfg(**kw)
    views = [q or _view(4, 100), k or _view(2, 300), v or _view(2, 300), out or _view(4, 100)]
    return B.load_library().httm_attention_forward(cfg, *views, lse, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), ARG), (dict(q_len=-1), ARG), (dict(kv_len=-2), ARG), (dict(heads=0), ARG), (dict(kv_heads=0), ARG),
    (dict(heads=5), ARG), (dict(d_head=0), ARG), (dict(dtype=7), ARG), (dict(softmax_scale=-1.0), ARG),
    (dict(softmax_scale=float("nan")), ARG), (dict(softmax_scale=float("inf")), ARG),
    (dict(softmax_scale=1e-30), ARG), (dict(softmax_scale=1e30), ARG),
    (dict(dtype=1), UNSUPPORTED), (dict(d_head=72), UNSUPPORTED), (dict(d_head=12), UNSUPPORTED),
    (dict(q_len=(1 << 21) + 1), UNSUPPORTED), (dict(kv_len=(1 << 30) + 1), UNSUPPORTED),
    (dict(batch=40000), UNSUPPORTED), (dict(batch=1, heads=2000, kv_heads=1, q_len=1 << 21), UNSUPPORTED),
])
def test_attention_shapes(kw, status):
    assert _forward(**kw) == status
    assert B.load_library().httm_attention_workspace_bytes(_cfg(**kw), None, None) == status


def test_attention_pointers_strides_and_workspace():
    lib = B.load_library()
    null = ctypes.c_void_p(None)
    assert lib.httm_attention_forward(None, null, null, null, null, None, None, 0, None) == ARG
    assert lib.httm_attention_forward(_cfg(), null, null, null, null, None, None, 0, None) == ARG
    assert _forward(q=_view(4, 100, data=0)) == ARG
    assert _forward(q=_view(4, 100, data=FAKE + 8)) == ALIGN
    assert _forward(k=_view(2, 300, token=68)) == ALIGN
    assert _forward(v=_view(2, 300, head=-64)) == ARG
    assert _forward(v=_view(2, 300, token=0)) == ARG                    # tokens cannot be broadcast
    assert _forward(out=_view(4, 100, head=0)) == ARG                   # an output that overlaps itself
    assert _forward(out=_view(4, 100, token=32)) == ARG
    assert _forward(out=_view(4, 100, batch=64 * 100)) == ARG
    assert _forward(lse=FAKE + 2) == ALIGN
    assert _forward(key_end=FAKE + 1) == ALIGN
    # keys split over the SMs: the partial sums need a workspace
    need = ops.httm_attention_workspace_bytes(2, 4, 2, 100, 8000, 64)[0]
    assert need > 0
    assert _forward(kv_len=8000) == WORKSPACE
    assert _forward(kv_len=8000, ws=None, n=need) == WORKSPACE
    assert _forward(kv_len=8000, n=need - 1) == WORKSPACE
    assert _forward(kv_len=8000, ws=FAKE + 16, n=need) == ALIGN
    # nothing to do
    assert _forward(batch=0) == 0
    assert _forward(q_len=0, q=_view(4, 0, data=0), out=_view(4, 0, data=0)) == 0

    def backward(ws=FAKE, n=0, lse=FAKE, **kw):
        q, k = _view(4, 100), _view(2, 300)
        views = [kw.get(x, y) for x, y in (("dout", q), ("q", q), ("k", k), ("v", k), ("out", q))]
        grads = [kw.get(x, y) for x, y in (("dq", q), ("dk", k), ("dv", k))]
        return lib.httm_attention_backward(_cfg(), *views, lse, *grads, ws, n, None)

    assert backward() == WORKSPACE
    assert backward(ws=None, n=1 << 40) == WORKSPACE
    assert backward(lse=None) == ARG
    assert backward(dk=_view(2, 300, head=0)) == ARG
    assert backward(dout=_view(4, 100, data=FAKE + 2)) == ALIGN


def test_attention_workspace_is_a_function_of_the_sizes():
    f, b = ops.httm_attention_workspace_bytes(1, 1, 1, 1, 41070, 64)
    assert f > 0 and f % 4 == 0
    assert ops.httm_attention_workspace_bytes(0, 16, 16, 1, 1369, 64) == (0, 0)
    # at least lse and D of every query row and head, and every row's range
    b = ops.httm_attention_workspace_bytes(30, 16, 16, 1369, 1369, 64)[1]
    assert 30 * 1369 * (16 * 8 + 8) <= b <= 30 * 1536 * (16 * 64 + 64)


def _rot(**kw):
    a = dict(batch=2, tokens=10, heads=4, kv_heads=2, d_head=64, dtype=0, axes=2, pairs=16, layout=0, inverse=0,
             factor=1.0, positions=FAKE, position_batch=20, freqs=FAKE)
    a.update(kw)
    return ops.httm_rotary_cfg(*a.values())


def _rotary(q=None, q_out=None, k=None, k_out=None, **kw):
    views = [q or _view(4, 10), q_out or _view(4, 10), k or _view(2, 10), k_out or _view(2, 10)]
    return B.load_library().httm_rotary(_rot(**kw), *views, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), ARG), (dict(tokens=-1), ARG), (dict(heads=0), ARG), (dict(kv_heads=-1), ARG), (dict(d_head=0), ARG),
    (dict(axes=0), ARG), (dict(axes=5), ARG), (dict(pairs=0), ARG), (dict(pairs=17), ARG), (dict(layout=2), ARG),
    (dict(dtype=2), ARG), (dict(factor=float("nan")), ARG), (dict(position_batch=-1), ARG), (dict(positions=0), ARG),
    (dict(freqs=0), ARG), (dict(freqs=FAKE + 4), ALIGN), (dict(positions=FAKE + 2), ALIGN),
    (dict(d_head=1025), UNSUPPORTED), (dict(tokens=0), 0), (dict(batch=0), 0),
    (dict(q=ops.httm_view(FAKE + 1, 2560, 640, 64)), ALIGN), (dict(q=ops.httm_view(0, 2560, 640, 64)), ARG),
    (dict(q_out=ops.httm_view(FAKE, 2560, 0, 64)), ARG), (dict(k=ops.httm_view(FAKE, -64, 640, 64)), ARG),
])
def test_rotary_arguments(kw, status):
    assert _rotary(**kw) == status


def _norm(**kw):
    a = dict(rows=12, channels=64, stream_dtype=0, branch_dtype=0, post=0, pre=1, gates=1, post_eps=1e-5, pre_eps=1e-5,
             residual_scale=1.0)
    a.update(kw)
    return ops.httm_norm_cfg(*a.values())


def _rows(data=FAKE, row=64):
    return ops.httm_rows(data, row)


def _gated(x=None, f=True, y=True, z=True, gate=FAKE, w=None, **kw):
    w = w or ops.httm_norm_weights(gate or 0, 0, 0, 0, 0)
    pick = lambda t: _rows() if t is True else t  # noqa: E731
    return B.load_library().httm_gated_norm_forward(_norm(**kw), w, x or _rows(), pick(f), pick(y), pick(z),
                                                    FAKE, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), ARG), (dict(channels=0), ARG), (dict(gates=-1), ARG), (dict(gates=5), ARG), (dict(stream_dtype=3), ARG),
    (dict(branch_dtype=-1), ARG), (dict(post=3), ARG), (dict(pre=-1), ARG), (dict(pre_eps=-1.0), ARG),
    (dict(post_eps=float("nan")), ARG), (dict(residual_scale=float("inf")), ARG), (dict(channels=8193), UNSUPPORTED),
    (dict(gates=1025, rows=2050), UNSUPPORTED), (dict(rows=1 << 31, gates=1), UNSUPPORTED),
    (dict(branch_dtype=1), UNSUPPORTED), (dict(pre=0), ARG), (dict(z=None), ARG), (dict(gate=None), ARG),
    (dict(gates=0), ARG), (dict(f=None), ARG), (dict(y=None), ARG), (dict(f=None, y=None, gates=0, gate=None, residual_scale=2.0), ARG),
    (dict(x=_rows(FAKE + 1)), ALIGN), (dict(x=_rows(0)), ARG), (dict(y=_rows(FAKE, 63)), ARG), (dict(z=_rows(FAKE, 0)), ARG),
    (dict(w=ops.httm_norm_weights(FAKE, 0, 0, FAKE + 2, 0)), ALIGN), (dict(rows=0), 0),
])
def test_gated_norm_arguments(kw, status):
    assert _gated(**kw) == status


def test_gated_norm_backward_arguments():
    lib = B.load_library()

    def call(cfg=None, w=None, dy=_rows(), dz=_rows(), f=_rows(), y=_rows(), stats=FAKE, dx=_rows(), df=_rows(),
             grads=None, ws=None, n=0):
        w = w or ops.httm_norm_weights(FAKE, 0, 0, 0, 0)
        g = grads or ops.httm_norm_grads(FAKE, 0, 0, 0, 0)
        return lib.httm_gated_norm_backward(cfg or _norm(), w, dy, dz, f, y, stats, dx, df, g, ws, n, None)

    assert call() == WORKSPACE
    need = ctypes.c_size_t(0)
    assert lib.httm_gated_norm_workspace_bytes(_norm(), R(need)) == 0 and need.value > 0
    assert lib.httm_gated_norm_workspace_bytes(_norm(), None) == ARG
    assert call(ws=FAKE + 4, n=1 << 30) == ALIGN
    assert call(dz=None) == ARG
    assert call(y=None) == ARG
    assert call(stats=None) == ARG
    assert call(f=None) == ARG
    assert call(grads=ops.httm_norm_grads(0, FAKE, 0, 0, 0)) == ARG     # no post norm to have a gradient
    assert call(dx=_rows(FAKE, 10)) == ARG
    assert call(w=ops.httm_norm_weights(0, 0, 0, 0, 0)) == ARG


def test_python_refuses_tensors_before_the_call():
    q = torch.zeros((2, 4, 8, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.httm_attention_forward(q, q, q)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.httm_attention_backward(q, q, q, q, q, q[..., 0])
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.httm_rotary(q, None, torch.ones(32, dtype=torch.float64), torch.zeros(8, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.httm_gated_norm_forward(torch.zeros(4, 64), pre=ops.Norm(ops.HTTM_NORM_LAYER))
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.httm_gated_norm_backward(None, torch.zeros(4, 64), None, torch.zeros(4, 64), torch.zeros(4, 4),
                                     pre=ops.Norm(ops.HTTM_NORM_LAYER))


def test_ranges_and_frequencies_on_the_host():
    b, e = ops.causal_ranges(2, 3, 5, device="cpu")
    assert b.tolist() == [[0, 0, 0]] * 2 and e.tolist() == [[3, 4, 5]] * 2
    b, e = ops.causal_ranges(1, 4, 4, window=2, device="cpu")
    assert b.tolist() == [[0, 0, 1, 2]] and e.tolist() == [[1, 2, 3, 4]]
    b, e = ops.causal_ranges(1, 4, 2, device="cpu")                # more queries than keys: the first see nothing
    assert e.tolist() == [[0, 0, 1, 2]]
    assert ops.frame_ranges(1, 4, 6, 3, device="cpu")[1].tolist() == [[3, 6, 6, 6]]
    assert ops.length_ranges(torch.tensor([2, 0]), 2)[1].tolist() == [[2, 2], [0, 0]]
    f, factor = ops.rotary_frequencies(4, base=10000.0, device="cpu")
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-15) and factor == 1.0
    assert torch.equal(ops.rotary_frequencies(4, scaling="linear", scale=4.0, device="cpu")[0], f / 4)
    n = ops.rotary_frequencies(4, scaling="ntk", scale=8.0, device="cpu")[0]
    assert n[0] == 1.0 and abs(float(n[3] * 8 / f[3]) - 1) < 1e-12   # the fastest kept, the slowest interpolated
    y, factor = ops.rotary_frequencies(64, scaling="yarn", scale=8.0, device="cpu")
    full = ops.rotary_frequencies(64, device="cpu")[0]
    assert y[0] == full[0] and abs(float(y[-1] * 8 / full[-1]) - 1) < 1e-12 and factor > 1
    with pytest.raises(ValueError):
        ops.rotary_frequencies(4, scaling="cubic", device="cpu")


@pytest.mark.parametrize("batch,heads,kv_heads,q_len,kv_len", [
    (16, 1, 1, 1, 8192), (4, 16, 4, 1, 8192), (64, 1, 1, 1, 32768), (1, 16, 16, 1, 1369), (1, 16, 16, 2, 4000),
    (1, 2, 2, 60, 4000), (3, 8, 1, 4, 100000), (1, 1, 1, 33, 9000)])
def test_attention_workspace_depends_on_the_extents_alone(batch, heads, kv_heads, q_len, kv_len):
    """The same bytes with key ranges and without, so that a workspace sized
    from the extents serves both."""
    args = (batch, heads, kv_heads, q_len, kv_len, 64)
    plain = ops.httm_attention_workspace_bytes(*args)
    for begin, end in ((0, FAKE), (FAKE, 0), (FAKE, FAKE)):
        assert ops._attention_bytes(ops.httm_attention(*args, 0, 0.0, begin, end)) == plain


def test_package_imports_on_a_torch_without_cuda():
    """Host-only use (planning, sizes) needs none of torch's CUDA bindings."""
    code = ("import torch\n"
            "for n in [n for n in dir(torch._C) if n.startswith('_cuda_')]: delattr(torch._C, n)\n"
            "import token_merging_view_b200 as p\n"
            "assert p.httm_attention_workspace_bytes(1, 2, 2, 100, 100, 64)[1] > 0\n"
            "assert p.causal_ranges(1, 2, 2, device='cpu')[1].tolist() == [[1, 2]]\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("device,index", [(None, 3), ("cuda", 3), (torch.device("cuda"), 3), ("cuda:1", 1), (0, 0),
                                          (torch.device("cuda", 2), 2)])
def test_device_status_reads_the_device_that_is_meant(device, index, monkeypatch):
    class Seen(Exception):
        pass

    def on(i, stream):
        raise Seen(i)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(ops, "_On", on)
    with pytest.raises(Seen) as seen:
        ops.httm_ops_device_status(device)
    assert seen.value.args == (index,)


@pytest.mark.parametrize("ns", [-1, 2 ** 64])
def test_wait_budget_is_within_64_bits(ns):
    with pytest.raises(ValueError, match="nanoseconds"):
        ops.httm_ops_set_wait_budget(ns)
