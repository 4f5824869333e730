"""The norms before and after a block, with gate and residual, against their
definition in 64 bits, forward and backward.  The norm before the next block
is defined on the stream as it is stored, so it is checked on the kernel's
own y."""
from __future__ import annotations

import pytest
import torch

import oplib
from oplib import FN
from token_merging_view_b200 import ops

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NONE, LAYER, RMS = ops.HTTM_NORM_NONE, ops.HTTM_NORM_LAYER, ops.HTTM_NORM_RMS


def _rand(shape, seed, dtype=F32, scale=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale + mean).to(dtype)


def _half_step(dtype):
    return oplib.U if dtype == BF else 2.0 ** -24


def _params(kind, C, seed, weight=True, bias=True):
    if kind == NONE:
        return None
    return ops.Norm(kind, _rand((C,), seed, scale=0.3, mean=1.0) if weight else None,
                    _rand((C,), seed + 1, scale=0.3) if bias else None, eps=1e-5)


def _w(t, C, fill):
    return torch.full((C,), float(fill), dtype=torch.float64, device="cuda") if t is None else t.double()


def _reference(x, f, gate, post, pre, rs, y, dy, dz):
    """Every output in 64 bits with its bound.  FN bounds fp32 chains of
    fewer than 128 additions; a result of storage type is rounded once."""
    R, C = x.shape
    res, tol = {}, {}
    g = 1.0 if gate is None else gate.double().view(-1, C).repeat_interleave(R // gate.view(-1, C).shape[0], 0)
    a = e_a = torch.zeros((R, C), dtype=torch.float64, device="cuda")
    if f is not None:
        a = f.double()
        if post is not None:
            n, r, e_n = oplib.normal(a, post.kind, post.eps)
            pw, pb = _w(post.weight, C, 1), _w(post.bias, C, 0)
            a, e_a = n * pw + pb, e_n * pw.abs() + FN * (n * pw).abs() + FN * pb.abs()
    y64 = rs * x.double() + g * a
    e_y = g.abs() * (e_a + FN * a.abs()) if gate is not None else e_a + FN * a.abs()
    res["y"], tol["y"] = y64, e_y + FN * (rs * x.double()).abs() + _half_step(x.dtype) * (y64.abs() + e_y)
    y = y.double()
    if pre is not None:
        hat, rr, e_hat = oplib.normal(y, pre.kind, pre.eps)
        w, b = _w(pre.weight, C, 1), _w(pre.bias, C, 0)
        z = hat * w + b
        e_z = e_hat * w.abs() + FN * (z.abs() + b.abs())
        bdt = f.dtype if f is not None else x.dtype
        res["z"], tol["z"] = z, e_z + _half_step(bdt) * (z.abs() + e_z)
    if dy is None and dz is None:
        return res, tol
    G = torch.zeros((R, C), dtype=torch.float64, device="cuda") if dy is None else dy.double()
    e_G = torch.zeros_like(G)
    # partial sums run over at most 128 rows a thread, then fewer than 100 additions
    FS = 2 * FN
    if pre is not None:
        u = dz.double()
        res["dpre_weight"] = (u * hat).sum(0)
        tol["dpre_weight"] = (u.abs() * (e_hat + FS * hat.abs())).sum(0)
        res["dpre_bias"], tol["dpre_bias"] = u.sum(0), FS * u.abs().sum(0)
        v, e_v = oplib.normal_grad(u * w, hat, rr, e_hat, pre.kind)
        G, e_G = G + v, e_v + FN * (G.abs() + v.abs())
    res["dx"] = rs * G
    tol["dx"] = abs(rs) * (e_G + FN * G.abs()) + _half_step(x.dtype) * (res["dx"].abs() + abs(rs) * e_G)
    if f is not None:
        if gate is not None:
            per = lambda t: t.view(gate.view(-1, C).shape[0], -1, C).sum(1)  # noqa: E731
            res["dgate"] = per(G * a)
            tol["dgate"] = per(e_G * (a.abs() + e_a) + G.abs() * (e_a + FS * a.abs()))
        ga = torch.as_tensor(g, dtype=torch.float64, device="cuda").abs()
        df, e_df = G * g, ga * (e_G + FN * G.abs())
        if post is not None:
            res["dpost_weight"] = (df * n).sum(0)
            tol["dpost_weight"] = (e_df * (n.abs() + e_n) + df.abs() * (e_n + FS * n.abs())).sum(0)
            res["dpost_bias"], tol["dpost_bias"] = df.sum(0), (e_df + FS * df.abs()).sum(0)
            u, e_u = df * pw, e_df * pw.abs()
            df, e2 = oplib.normal_grad(u, n, r, e_n, post.kind)
            _, e3 = oplib.normal_grad(e_u / FN, n, r, e_n, post.kind)       # the input's own bound, carried through
            e_df = e2 + e3
        res["df"], tol["df"] = df, e_df + _half_step(f.dtype) * (df.abs() + e_df)
    return res, tol


def _run(x, f, gate, post, pre, rs, dy, dz, **kw):
    how = dict(gate=gate, post=post, pre=pre, residual_scale=rs)
    y, z, stats = ops.httm_gated_norm_forward(x, f, **how, **kw)
    got = dict(y=y, z=z)
    grads = ops.httm_gated_norm_backward(dy, dz, f, y, stats, **how)
    return {k: t for k, t in {**got, **grads}.items() if t is not None}


def _compare(R, C, stream, branch, post, pre, gates, rs=1.0, seed=0, with_dy=True, weight=True, bias=True):
    x, f = _rand((R, C), seed, stream, 2.0, 0.3), _rand((R, C), seed + 1, branch, 1.0, 0.1)
    gate = _rand((gates, C), seed + 2, scale=0.5) if gates else None
    post, pre = _params(post, C, seed + 3, weight, bias), _params(pre, C, seed + 5, weight, bias)
    dy = _rand((R, C), seed + 7, stream) if with_dy else None
    dz = _rand((R, C), seed + 8, branch) if pre is not None else None
    got = _run(x, f, gate, post, pre, rs, dy, dz)
    want, tol = _reference(x, f, gate, post, pre, rs, got["y"], dy, dz)
    missing = {"dpre_weight", "dpre_bias", "dpost_weight", "dpost_bias"} - set(got)
    for name in want:
        if name in missing:
            continue                                       # a norm without that parameter has no such gradient
        oplib.check(got[name], want[name], tol[name], name)
    return got


CASES = [
    # rows, channels, stream, branch, post, pre, gates, residual_scale
    (1, 1, F32, F32, NONE, RMS, 1, 1.0),
    (1, 1024, BF, BF, NONE, LAYER, 1, 1.0),
    (37, 1024, BF, BF, NONE, LAYER, 1, 1.0),
    (300, 1024, BF, BF, LAYER, LAYER, 3, 0.5),
    (64, 1024, F32, BF, RMS, RMS, 0, 1.0),
    (5, 7, BF, BF, LAYER, RMS, 5, 1.0),
    (129, 250, F32, F32, RMS, LAYER, 1, -2.0),
    (77, 264, BF, BF, NONE, RMS, 7, 1.0),
    (50, 513, F32, BF, LAYER, NONE, 2, 1.0),
    (66, 1001, BF, BF, RMS, RMS, 2, 0.0),
    (40, 2048, BF, BF, NONE, LAYER, 1, 1.0),
    (9, 4100, F32, F32, LAYER, LAYER, 3, 1.0),
    (8, 8192, BF, BF, RMS, LAYER, 1, 1.0),
    (6, 8191, F32, BF, NONE, RMS, 2, 1.0),
    (1024, 16, BF, BF, NONE, LAYER, 1024, 1.0),
    (4000, 40, BF, BF, LAYER, NONE, 0, 1.0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_against_definition(case):
    _compare(*case)


@pytest.mark.parametrize("post", [NONE, LAYER])
@pytest.mark.parametrize("C", [256, 257, 512, 1032, 2048, 2049, 2050, 3016, 4096, 4097])
def test_channels_a_thread(C, post):
    """Both sides of every change in the threads a row takes, with more rows
    than the GPU holds at a time and odd, paired and whole accesses."""
    _compare(2500, C, BF, BF, post, LAYER, 2)


def test_without_parameters_or_stream_gradient():
    _compare(33, 96, BF, BF, RMS, LAYER, 1, weight=False, bias=False)
    _compare(33, 96, F32, BF, NONE, RMS, 0, bias=False, with_dy=False)
    # nothing multiplies the threads behind the row's end by a weight of 0
    for C in (2, 24, 150, 315, 1030, 5000):
        _compare(9, C, F32, F32, LAYER, LAYER, 0, weight=False, bias=False)


def test_norm_before_a_first_block():
    """No block output: z = pre(x), y is x itself; its backward call takes x."""
    x, dz, dy = _rand((90, 520), 1, F32, 3.0), _rand((90, 520), 2, BF), _rand((90, 520), 3, F32)
    pre = _params(LAYER, 520, 4)
    y, z, stats = ops.httm_gated_norm_forward(x, pre=pre, branch_dtype=BF)
    assert y is x and z.dtype == BF
    got = ops.httm_gated_norm_backward(dy, dz, None, y, stats, pre=pre)
    want, tol = _reference(x, None, None, None, pre, 1.0, x, dy, dz)
    e = tol["z"] + oplib.U * want["z"].abs()               # z is stored in bf16 here
    oplib.check(z, want["z"], e, "z")
    for n in ("dx", "dpre_weight", "dpre_bias"):
        oplib.check(got[n], want[n], tol[n], n)
    assert got["df"] is None and got["dgate"] is None
    y2, z2, _ = ops.httm_gated_norm_forward(x, pre=pre, branch_dtype=BF, residual_scale=2.0)
    assert torch.equal(y2, 2 * x) and z2.dtype == BF


def test_large_mean_keeps_the_variance():
    """Rows whose mean is 1000 times their deviation: the squares are taken
    after the mean, so the variance keeps its digits."""
    x, f = _rand((20, 1024), 1, F32, 0.5, 500.0), torch.zeros((20, 1024), device="cuda")
    pre = ops.Norm(LAYER, eps=1e-6)
    y, z, _ = ops.httm_gated_norm_forward(x, f, pre=pre)
    hat, _, e = oplib.normal(x.double(), LAYER, 1e-6)
    assert torch.equal(y, x)
    # here the mean's own error, FN 500, is what counts: below 1e-2 of a deviation
    assert (z.double() - hat).abs().max() <= float(e.max())
    assert (z.double() - hat).abs().max() <= 2.0 ** -17 * 500 / 0.5


def test_strides_in_place_and_same_bits():
    R, C = 70, 1024
    x, f = _rand((R, C), 1, BF), _rand((R, C), 2, BF)
    gate, pre, post = _rand((2, C), 3), _params(LAYER, C, 4), _params(RMS, C, 6)
    dy, dz = _rand((R, C), 8, BF), _rand((R, C), 9, BF)
    want = _run(x, f, gate, post, pre, 1.0, dy, dz)
    for _ in range(3):
        again = _run(x, f, gate, post, pre, 1.0, dy, dz)
        for n in want:
            assert torch.equal(want[n], again[n]), n
    # rows apart on 16 bytes: the same accesses, the same bits; rows off 16
    # bytes: element accesses, which add a row up in another order
    for width, at in ((2 * C + 8, 8), (2 * C + 3, 0), (2 * C + 3, 3)):
        s = []
        for t in (x, f):
            b = torch.zeros((R, width), dtype=BF, device="cuda")
            b[:, at:at + C] = t
            s.append(b[:, at:at + C])
        how = dict(gate=gate, post=post, pre=pre)
        y, z, stats = ops.httm_gated_norm_forward(s[0], s[1], y=s[0], **how)      # the stream in place
        assert y.data_ptr() == s[0].data_ptr()
        g = ops.httm_gated_norm_backward(dy, dz, s[1], y, stats, **how)
        got = {**dict(y=y, z=z), **g}
        exact, tol = _reference(x, f, gate, post, pre, 1.0, y, dy, dz)
        for n in want:
            if width % 8 == 0:
                assert torch.equal(got[n], want[n]), n
            else:
                oplib.check(got[n], exact[n], tol[n], n)
    dx = dy.clone()
    y, z, stats = ops.httm_gated_norm_forward(x, f, gate=gate, post=post, pre=pre)
    g = ops.httm_gated_norm_backward(dx, dz, f, y, stats, gate=gate, post=post, pre=pre, dx=dx)
    assert torch.equal(dx, want["dx"]) and g["dx"] is dx


def test_rows_of_one_do_not_reach_another():
    R, C = 40, 300
    x, f = _rand((R, C), 1, F32), _rand((R, C), 2, F32)
    pre, post = _params(LAYER, C, 3), _params(LAYER, C, 5)
    dy, dz = _rand((R, C), 7, F32), _rand((R, C), 8, F32)
    want = _run(x, f, None, post, pre, 1.0, dy, dz)
    x[5], f[9], dz[11] = float("nan"), float("inf"), float("nan")
    got = _run(x, f, None, post, pre, 1.0, dy, dz)
    keep = torch.ones(R, dtype=torch.bool, device="cuda")
    keep[[5, 9, 11]] = False
    for n in ("y", "z", "dx", "df"):
        assert torch.equal(got[n][keep], want[n][keep]), n
    assert torch.isnan(got["z"][5]).all() and torch.isnan(got["z"][9]).all()


def test_no_rows_graph_and_stream():
    C = 128
    pre, gate = _params(LAYER, C, 1), _rand((C,), 3)
    e = torch.empty((0, C), device="cuda")
    got = _run(e, e, gate, None, pre, 1.0, e, e)
    assert got["y"].shape == (0, C)
    for n in ("dgate", "dpre_weight", "dpre_bias"):
        assert got[n].shape == (C,) and (got[n] == 0).all()
    x, f, dy, dz = (_rand((33, C), s, BF) for s in range(4))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = _run(x, f, gate, None, pre, 1.0, dy, dz)
    for t in (x, f, dy, dz):
        t.mul_(-0.5)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    want = _run(x, f, gate, None, pre, 1.0, dy, dz)
    for n in want:
        assert torch.equal(got[n], want[n]), n


def test_gradients_against_differences():
    R, C = 12, 40
    x, f = _rand((R, C), 1, F32), _rand((R, C), 2, F32)
    gate, post, pre = _rand((3, C), 3), _params(LAYER, C, 4), _params(RMS, C, 6)
    dy, dz = _rand((R, C), 8, F32), _rand((R, C), 9, F32)
    got = _run(x, f, gate, post, pre, 0.7, dy, dz)
    leaves = dict(dx=x, df=f, dgate=gate, dpost_weight=post.weight, dpost_bias=post.bias, dpre_weight=pre.weight,
                  dpre_bias=pre.bias)

    def loss(v):
        n, _, _ = oplib.normal(v["df"], LAYER, post.eps)
        a = n * v["dpost_weight"] + v["dpost_bias"]
        y = 0.7 * v["dx"] + v["dgate"].repeat_interleave(R // 3, 0) * a
        h, _, _ = oplib.normal(y, RMS, pre.eps)
        z = h * v["dpre_weight"] + v["dpre_bias"]
        return (y * dy.double()).sum() + (z * dz.double()).sum()

    base = {n: t.double() for n, t in leaves.items()}
    _, tol = _reference(x, f, gate, post, pre, 0.7, got["y"], dy, dz)
    for i, name in enumerate(leaves):
        u = torch.randn(base[name].shape, dtype=torch.float64, device="cuda",
                        generator=torch.Generator(device="cuda").manual_seed(i))
        h = 1e-6
        want = (loss({**base, name: base[name] + h * u}) - loss({**base, name: base[name] - h * u})) / (2 * h)
        bound = (u.abs() * tol[name]).sum() + 1e-6 * (1 + want.abs())
        # y is stored in fp32: its rounding moves the rows that the norm reads by 2^-24
        bound = bound + 2.0 ** -20 * (u.abs() * got[name].double().abs()).sum()
        assert ((got[name].double() * u).sum() - want).abs() <= bound, name


def test_refusals():
    x = torch.zeros((12, 64), device="cuda")
    n = ops.Norm(LAYER)
    for bad in (dict(x=x.half()), dict(x=x[0]), dict(x=x.t().contiguous().t()), dict(f=x.bfloat16(), x=x.bfloat16(), z=x),
                dict(f=x[:5]), dict(gate=torch.zeros(63, device="cuda")), dict(gate=torch.zeros((5, 64), device="cuda")),
                dict(gate=torch.zeros(64, dtype=BF, device="cuda")), dict(pre=ops.Norm(LAYER, torch.zeros(63, device="cuda"))),
                dict(pre=ops.Norm(LAYER, torch.zeros(64))), dict(z=x.bfloat16()), dict(pre=None, z=x), dict(y=x[:, :1].expand(12, 64)),
                dict(stats=torch.zeros((4, 11), device="cuda")), dict(f=None, gate=torch.zeros(64, device="cuda")),
                dict(x=x.bfloat16(), f=x), dict(pre=ops.Norm(5)), dict(pre=ops.Norm(LAYER, eps=-1.0))):
        with pytest.raises((ValueError, ops.HttmError)):
            ops.httm_gated_norm_forward(**{**dict(x=x, f=x, pre=n), **bad})
    y, z, stats = ops.httm_gated_norm_forward(x, x, pre=n)
    for bad in (dict(dz=None), dict(dz=z[:4]), dict(stats=stats[:2]), dict(dy=z.bfloat16()), dict(f=None, df=x),
                dict(workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"), pre=ops.Norm(LAYER, torch.ones(64, device="cuda")))):
        with pytest.raises((ValueError, ops.HttmError)):
            ops.httm_gated_norm_backward(**{**dict(dy=x, dz=z, f=x, y=y, stats=stats, pre=n), **bad})
