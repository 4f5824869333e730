"""Attention over key ranges against its definition in 64 bits: forward and
gradients, at the lengths, masks, head layouts and strides where tiles,
splits and packing can go wrong.  The bounds (tests/oplib.py) follow from the
roundings to bf16 and the fp32 sums."""
from __future__ import annotations

import pytest
import torch

import oplib
from token_merging_view_b200 import ops

pytestmark = pytest.mark.gpu


def _rand(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).bfloat16()


def _inputs(B, H, K, L, N, d, seed=0):
    return (_rand((B, H, L, d), seed), _rand((B, K, N, d), seed + 1), _rand((B, K, N, d), seed + 2),
            _rand((B, H, L, d), seed + 3))


def _ranges(mask, B, L, N, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 77)
    if mask == "none":
        return None, None
    if mask == "causal":
        return ops.causal_ranges(B, L, N)
    if mask == "window":
        return ops.causal_ranges(B, L, N, window=37)
    if mask == "frames":
        return ops.frame_ranges(B, L, N, 50)
    if mask == "padded":                       # lengths from 0 up; the queries behind them see nothing
        n = torch.randint(0, N + 1, (B,), generator=g, device="cuda")
        n[0] = N
        if B > 1:
            n[-1] = 0
        b, e = ops.length_ranges(n, L)
        e[torch.arange(L, device="cuda")[None] >= n[:, None] + (L - N if L > N else 0)] = 0
        return b, e
    if mask == "packed":                       # sequences side by side: block-diagonal
        cut = torch.sort(torch.randint(0, L + 1, (3,), generator=g, device="cuda")).values.tolist()
        b, e = torch.zeros((B, L), dtype=torch.int32, device="cuda"), torch.zeros((B, L), dtype=torch.int32, device="cuda")
        for s, t in zip([0] + cut, cut + [L]):
            b[:, s:t], e[:, s:t] = s, t
        return b, e
    assert mask == "random"                    # any pair: empty, reversed, below 0, above N
    b = torch.randint(-5, N + 5, (B, L), generator=g, device="cuda").int()
    e = torch.randint(-5, N + 5, (B, L), generator=g, device="cuda").int()
    return b, e


def _run(q, k, v, dout, b, e, **kw):
    out, lse = ops.httm_attention_forward(q, k, v, b, e, **kw)
    dq, dk, dv = ops.httm_attention_backward(dout, q, k, v, out, lse, b, e, **kw)
    assert ops.httm_ops_device_status() == 0
    return dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv)


def _compare(q, k, v, dout, b, e, **kw):
    got = _run(q, k, v, dout, b, e, **kw)
    want, tol = oplib.attention(q, k, v, b, e, dout, kw.get("softmax_scale"))
    for name in want:
        oplib.check(got[name], want[name], tol[name], name)
    return got


CASES = [
    # B, H, K, L, N, d, mask
    (1, 1, 1, 1, 1, 64, "none"),
    (1, 1, 1, 1, 1, 8, "causal"),
    (1, 2, 1, 1, 129, 64, "none"),
    (2, 4, 2, 3, 300, 40, "padded"),
    (1, 2, 2, 128, 128, 64, "causal"),
    (1, 3, 1, 127, 129, 8, "causal"),
    (2, 2, 2, 129, 129, 64, "window"),
    (2, 2, 1, 257, 257, 56, "frames"),
    (1, 6, 2, 300, 300, 64, "packed"),
    (2, 2, 2, 300, 700, 64, "random"),
    (3, 5, 5, 64, 65, 16, "padded"),
    (1, 8, 1, 100, 1000, 64, "window"),        # 8 heads packed: 800 rows against one key head
    (1, 7, 1, 300, 300, 24, "causal"),
    (4, 2, 2, 1, 515, 64, "padded"),
    (1, 16, 16, 5, 2000, 64, "causal"),        # keys split over the SMs
    (1, 2, 2, 700, 300, 64, "none"),           # more queries than keys
    (1, 1, 1, 1500, 1500, 64, "none"),         # queries of a key tile split
    (1, 2, 1, 513, 130, 64, "random"),
    # long enough for two groups of warps a block in dK/dV, dQ, or both
    (1, 2, 1, 1300, 1300, 64, "causal"),
    (1, 1, 1, 2500, 2500, 64, "window"),
    (2, 2, 2, 700, 3001, 40, "random"),
    (2, 4, 2, 1201, 3300, 64, "padded"),
    (1, 1, 1, 3500, 3500, 64, "packed"),
    # few rows a key head: one, 16, 17, 32 and (past them) 33
    (1, 1, 1, 1, 31, 64, "none"),
    (3, 16, 1, 1, 700, 64, "padded"),
    (2, 17, 1, 1, 700, 32, "random"),
    (2, 16, 1, 2, 9000, 64, "causal"),
    (2, 11, 1, 3, 400, 64, "random"),
    (5, 8, 2, 4, 333, 56, "window"),
    (1, 1, 1, 32, 32, 64, "packed"),
    (40, 8, 8, 1, 260, 64, "padded"),
    (1, 1, 1, 1, 20000, 64, "none"),           # one item: more parts than a cluster holds
    (1, 4, 2, 3, 5000, 64, "causal"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_against_definition(case):
    B, H, K, L, N, d, mask = case
    q, k, v, dout = _inputs(B, H, K, L, N, d)
    b, e = _ranges(mask, B, L, N)
    _compare(q, k, v, dout, b, e)


@pytest.mark.parametrize("case", [(37, 4, 4, 129, 8300, 64, "padded"), (37, 4, 2, 257, 8193, 24, "random"),
                                  (37, 4, 4, 129, 8192, 64, "random"), (37, 4, 4, 100, 97, 64, "padded"),
                                  (9, 4, 2, 700, 96, 64, "none"), (9, 4, 1, 301, 193, 40, "window")],
                         ids=lambda c: "-".join(map(str, c)))
def test_more_items_than_sms(case):
    """Enough rows that no keys are split: more than 8,192 keys and fewer, and
    steps of the keys that end at, before and behind a tile."""
    test_against_definition(case)


def test_scale_and_large_scores():
    """Scores far apart: the running maximum rises by more than 2^16 between
    tiles, and some probabilities underflow to 0."""
    q, k, v, dout = _inputs(1, 2, 2, 200, 600, 64)
    k = (k * torch.linspace(0.1, 6, 600, device="cuda")[None, None, :, None]).bfloat16()
    b, e = ops.causal_ranges(1, 200, 600)
    _compare(q, k, v, dout, b, e, softmax_scale=0.7)


@pytest.mark.parametrize("L,N", [(0, 5), (5, 0), (0, 0)])
def test_empty_lengths(L, N):
    q, k, v, dout = _inputs(2, 2, 1, L, N, 64)
    got = _run(q, k, v, dout, None, None)
    assert (got["out"] == 0).all() and (got["lse"] == -float("inf")).all()
    for n in ("dq", "dk", "dv"):
        assert (got[n] == 0).all()
    empty = ops.httm_attention_forward(q[:0], k[:0], v[:0])
    assert empty[0].shape == (0, 2, L, 64)


def test_three_dimensions_are_one_batch_entry():
    q, k, v, dout = _inputs(1, 4, 2, 77, 90, 64)
    a = _run(q, k, v, dout, None, None)
    b = _run(q[0], k[0], v[0], dout[0], None, None)
    for n in a:
        assert torch.equal(a[n][0], b[n])


def test_strided_inputs_and_outputs():
    """Views of a packed projection [B, L, 3, H, d] in, and a token-major
    output: the same bits as contiguous tensors."""
    B, H, L, d = 2, 3, 200, 48
    packed = _rand((B, L, 3, H, d), 5)
    q, k, v = (packed[:, :, i].transpose(1, 2) for i in range(3))
    dout = _rand((B, L, H, d), 6).transpose(1, 2)
    b, e = ops.causal_ranges(B, L, L)
    want = _run(*(t.contiguous() for t in (q, k, v, dout)), b, e)
    out = torch.empty((B, L, H, d), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    grads = torch.empty((B, L, 3, H, d), dtype=torch.bfloat16, device="cuda")
    dq, dk, dv = (grads[:, :, i].transpose(1, 2) for i in range(3))
    _, lse = ops.httm_attention_forward(q, k, v, b, e, out=out)
    ops.httm_attention_backward(dout, q, k, v, out, lse, b, e, dq=dq, dk=dk, dv=dv)
    for n, t in dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv).items():
        assert torch.equal(t, want[n]), n


def test_broadcast_inputs():
    """Keys and values shared over the batch and over heads (stride 0): the
    results, and the gradients of every copy, are those of repeated tensors."""
    B, H, K, L, N, d = 3, 4, 2, 70, 150, 64
    q, _, _, dout = _inputs(B, H, K, L, N, d)
    k0, v0 = _rand((1, 1, N, d), 8), _rand((1, K, N, d), 9)
    k, v = k0.expand(B, K, N, d), v0.expand(B, K, N, d)
    got = _run(q, k, v, dout, None, None)
    want = _run(q, k.contiguous(), v.contiguous(), dout, None, None)
    for n in want:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("H,L,N", [(4, 150, 300), (32, 150, 4000)])
def test_unseen_places_may_hold_anything(H, L, N):
    """NaN and infinities in keys and values nobody sees, and in queries,
    outputs and output gradients of rows that see nothing, change no bit."""
    B, K, d = 3, 2, 64
    q, k, v, dout = _inputs(B, H, K, L, N, d)
    n = torch.tensor([N, 129, 0], device="cuda")
    b, e = ops.length_ranges(n, L)
    b = b + torch.tensor([17, 0, 0], device="cuda", dtype=torch.int32)[:, None]
    e[1, 40:60] = 0
    want = _run(q, k, v, dout, b, e)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").bfloat16()
    j = torch.arange(N, device="cuda")
    unseen = (j[None] < b[:, :1]) | (j[None] >= n[:, None])
    q, k, v, dout = (t.clone() for t in (q, k, v, dout))
    fill = bad[torch.arange(d, device="cuda") % 3]
    for t in (k, v):
        t.copy_(torch.where(unseen[:, None, :, None], fill, t))
    none = (e <= b)[:, None, :, None]
    q, dout = torch.where(none, fill, q), torch.where(none, fill, dout)
    out, lse = ops.httm_attention_forward(q, k, v, b, e)
    assert torch.equal(out, want["out"]) and torch.equal(lse, want["lse"])
    out = torch.where(none, fill, out)
    grads = ops.httm_attention_backward(dout, q, k, v, out, lse, b, e)
    for name, t in zip(("dq", "dk", "dv"), grads):
        assert torch.equal(t, want[name]), name


def test_unseen_places_may_hold_anything_for_single_tokens():
    """A cache whose entries behind each sequence's length were never
    written, one sequence of length 0."""
    B, H, K, N, d = 4, 8, 2, 500, 64
    q, k, v, _ = _inputs(B, H, K, 1, N, d)
    n = torch.tensor([500, 33, 0, 257], device="cuda")
    b, e = ops.length_ranges(n, 1)
    want = ops.httm_attention_forward(q, k, v, b, e)
    unseen = (torch.arange(N, device="cuda")[None] >= n[:, None])[:, None, :, None]
    q = q.clone()
    q[2] = float("nan")
    for bad in (float("nan"), float("inf")):
        got = ops.httm_attention_forward(q, k.masked_fill(unseen, bad), v.masked_fill(unseen, bad), b, e)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (want[0][2] == 0).all() and (want[1][2] == -float("inf")).all()


def test_visible_nan_reaches_its_row():
    q, k, v, _ = _inputs(1, 1, 1, 10, 40, 64)
    q[0, 0, 3] = float("nan")
    out, lse = ops.httm_attention_forward(q, k, v)
    rows = torch.arange(10, device="cuda") != 3
    assert torch.isnan(out[0, 0, 3]).all() and torch.isnan(lse[0, 0, 3])
    assert torch.isfinite(out[0, 0, rows]).all() and torch.isfinite(lse[0, 0, rows]).all()


@pytest.mark.parametrize("G,L,N,mask", [(1, 300, 300, "causal"), (2, 300, 700, "random"), (1, 7, 90, "causal"),
                                        (4, 6, 1000, "random"), (1, 600, 5000, "window"), (1, 9, 20000, "random"),
                                        (1, 18900, 8300, "random")])
def test_values_reach_only_the_rows_that_see_them(G, L, N, mask):
    """Infinities and NaN in values (and NaN in keys) that some rows see and
    some do not: the others keep their bits, and those that see an infinity in
    a channel have it there."""
    K, d = 2, 64
    q, k, v, _ = _inputs(1, K * G, K, L, N, d)
    b, e = _ranges(mask, 1, L, N)
    want, lse = ops.httm_attention_forward(q, k, v, b, e)
    lo, hi = b.clamp(0, N)[0], e.clamp(0, N)[0]
    bad = {N - 1: float("nan"), N // 2: float("inf"), N // 3 + 1: -float("inf")}
    v = v.clone()
    for j, x in bad.items():
        v[:, :, j, j % d] = x
    out, lse2 = ops.httm_attention_forward(q, k, v, b, e)
    assert torch.equal(lse, lse2)
    for j, x in bad.items():
        c, sees = j % d, (lo <= j) & (j < hi)
        got = out[0, :, :, c].float()
        assert torch.equal(got[:, ~sees], want[0, :, ~sees, c].float()), j
        assert (torch.isnan(got[:, sees]) if x != x else got[:, sees] == x).all(), j
    rest = torch.ones(d, dtype=torch.bool, device="cuda")
    rest[[j % d for j in bad]] = False
    assert torch.equal(out[..., rest], want[..., rest])
    k = k.clone()
    k[:, :, N - 1] = float("nan")
    out, lse = ops.httm_attention_forward(q, k, v, b, e)
    sees = (lo <= N - 1) & (N - 1 < hi)
    assert torch.isnan(out[0, :, sees]).all() and torch.isnan(lse[0, :, sees]).all()
    assert torch.equal(lse[0, :, ~sees], lse2[0, :, ~sees])
    assert torch.equal(out[0][:, ~sees][..., rest], want[0][:, ~sees][..., rest])


def test_far_offsets():
    """Batch entries more than 2^31 elements apart (a long cache)."""
    N, d = 200, 64
    flat = torch.empty(2 ** 31 + 4 * N * d, dtype=torch.bfloat16, device="cuda")
    k = flat.as_strided((2, 1, N, d), (2 ** 31, 0, d, 1))
    v = flat[2 * N * d:].as_strided((2, 1, N, d), (2 ** 31, 0, d, 1))
    q, k0, v0, dout = _inputs(2, 2, 1, 33, N, d)
    k.copy_(k0)
    v.copy_(v0)
    got, want = _run(q, k, v, dout, None, None), _run(q, k0, v0, dout, None, None)
    for n in want:
        assert torch.equal(got[n], want[n]), n


def test_same_bits_every_time():
    q, k, v, dout = _inputs(1, 4, 1, 400, 900, 64)
    b, e = _ranges("random", 1, 400, 900)
    first = _run(q, k, v, dout, b, e)
    for _ in range(3):
        again = _run(q, k, v, dout, b, e)
        for n in first:
            assert torch.equal(first[n], again[n]), n


def test_captured_and_replayed():
    """Two graphs with their own workspaces, replayed on new inputs, give the
    eager bits; also when replayed at the same time on two streams."""
    B, H, K, L, N, d = 1, 4, 2, 140, 1300, 64
    b, e = ops.causal_ranges(B, L, N)
    sets = []
    for seed in (1, 50):
        q, k, v, dout = _inputs(B, H, K, L, N, d, seed)
        _run(q, k, v, dout, b, e)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out, lse = ops.httm_attention_forward(q, k, v, b, e)
            grads = ops.httm_attention_backward(dout, q, k, v, out, lse, b, e)
        sets.append((g, s, (q, k, v, dout), dict(zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)))))
    for _, _, ins, _ in sets:
        for t in ins:
            t.copy_(t.flip(-1) * 0.5)
    torch.cuda.synchronize()
    for g, s, _, _ in sets:
        with torch.cuda.stream(s):
            for _ in range(3):
                g.replay()
    torch.cuda.synchronize()
    for _, _, (q, k, v, dout), got in sets:
        want = _run(q, k, v, dout, b, e)
        for n in want:
            assert torch.equal(got[n], want[n]), n


def test_on_another_stream():
    q, k, v, dout = _inputs(2, 4, 4, 130, 600, 64)
    want = _run(q, k, v, dout, None, None)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = ops.httm_attention_forward(q, k, v, stream=s)
    grads = ops.httm_attention_backward(dout, q, k, v, out, lse, stream=s)
    s.synchronize()
    for n, t in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        assert torch.equal(t, want[n]), n


@pytest.mark.parametrize("L,N", [(9, 4000), (60, 4000), (1, 60000)])
def test_given_workspace_is_enough_and_checked(L, N):
    B, H, K, d = 1, 2, 2, 64
    q, k, v, dout = _inputs(B, H, K, L, N, d)
    want = _run(q, k, v, dout, None, None)
    need_f, need_b = ops.httm_attention_workspace_bytes(B, H, K, L, N, d)
    assert need_b > 0 and (need_f > 0 or L == 9)           # few rows on few keys need none
    guard = 4096
    ws = torch.full((max(need_f, need_b) + guard,), 0xA5, dtype=torch.uint8, device="cuda")
    out, lse = ops.httm_attention_forward(q, k, v, workspace=ws[:need_f])
    assert torch.equal(out, want["out"]) and (ws[need_f:] == 0xA5).all()
    ws.fill_(0xA5)
    grads = ops.httm_attention_backward(dout, q, k, v, out, lse, workspace=ws[:need_b])
    assert (ws[need_b:] == 0xA5).all()
    for n, t in zip(("dq", "dk", "dv"), grads):
        assert torch.equal(t, want[n]), n
    for call, need in ((lambda w: ops.httm_attention_forward(q, k, v, workspace=w), need_f),
                       (lambda w: ops.httm_attention_backward(dout, q, k, v, out, lse, workspace=w), need_b)):
        if need == 0:
            continue
        with pytest.raises(ops.HttmError) as err:
            call(ws[:need - 1])
        assert err.value.status == 4                      # HTTM_ERR_WORKSPACE


def test_rows_behind_the_outputs_are_left_alone():
    """Outputs inside larger buffers: nothing around them is written."""
    B, H, K, L, N, d = 1, 3, 1, 133, 260, 40
    q, k, v, dout = _inputs(B, H, K, L, N, d)
    bufs = {}
    for n, (h, t) in dict(out=(H, L), dq=(H, L), dk=(K, N), dv=(K, N)).items():
        bufs[n] = torch.full((B, h, t + 7, d + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    view = {n: t[:, :, :-7, :d] for n, t in bufs.items()}
    out, lse = ops.httm_attention_forward(q, k, v, out=view["out"])
    ops.httm_attention_backward(dout, q, k, v, out, lse, dq=view["dq"], dk=view["dk"], dv=view["dv"])
    want = _run(q, k, v, dout, None, None)
    for n, t in bufs.items():
        assert torch.equal(view[n], want[n]), n
        assert (t[:, :, -7:] == 3.0).all() and (t[..., d:] == 3.0).all(), n


def test_gradients_against_differences():
    """<gradient, direction> against central differences of the 64-bit
    forward; what the kernels may be off by is the bound of the gradients
    summed over the direction."""
    B, H, K, L, N, d = 1, 4, 2, 60, 60, 32
    q, k, v, dout = _inputs(B, H, K, L, N, d)
    b, e = ops.causal_ranges(B, L, N, window=20)
    got = _run(q, k, v, dout, b, e)
    _, tol = oplib.attention(q, k, v, b, e, dout)
    x = {"dq": q.double(), "dk": k.double(), "dv": v.double()}
    for i, name in enumerate(x):
        u = torch.randn(x[name].shape, dtype=torch.float64, device="cuda",
                        generator=torch.Generator(device="cuda").manual_seed(40 + i))
        h = 1e-5

        def loss(step):
            y = {n: t + step * u if n == name else t for n, t in x.items()}
            return (oplib.attention(y["dq"], y["dk"], y["dv"], b, e)[0]["out"] * dout.double()).sum()

        want = (loss(h) - loss(-h)) / (2 * h)
        bound = (u.abs() * tol[name]).sum() + 1e-6 * (1 + want.abs())
        assert ((got[name].double() * u).sum() - want).abs() <= bound, name


def test_agrees_with_the_dense_layer():
    """The dense layer (HTTM_DENSE) computes the same attention on [h, N, d]
    tensors: both within the bound of the definition."""
    from token_merging_view_b200 import binding as B
    h, T, P, d = 4, 2, 169, 64
    q, k, v, _ = _inputs(1, h, h, T * P, T * P, d)
    plan = B.httm_plan(B.LayerConfig(h=h, T=T, P=P, d_head=d, mode=B.HTTM_DENSE))
    dense = B.httm_forward(plan, q[0], k[0], v[0])
    out, _ = ops.httm_attention_forward(q[0], k[0], v[0])
    want, tol = oplib.attention(q, k, v)
    oplib.check(dense[None], want["out"], tol["out"], "dense")
    oplib.check(out[None], want["out"], tol["out"], "out")


@pytest.mark.parametrize("H,K,L,N,d,a,z", [
    (2, 2, 100, 300, 64, 10, 50),             # one tile of queries
    (4, 2, 300, 700, 40, 129, 131),           # several; the gap inside one step
    (8, 1, 2, 900, 64, 1, 899),               # few rows
    (1, 1, 2100, 2500, 64, 700, 1400),        # two groups of warps a block in dK/dV, whole steps in the gap
    (2, 1, 300, 3500, 64, 95, 3000),          # in dQ
    (1, 1, 2100, 3500, 24, 1000, 1100),       # in both
])
@pytest.mark.parametrize("order", ["halves", "in turn"])
def test_a_gap_between_ranges_may_hold_anything(H, K, L, N, d, a, z, order):
    """Queries of [0, a) beside queries of [z, N): NaN and infinities in the
    keys and values between, which nobody sees, change no bit."""
    q, k, v, dout = _inputs(1, H, K, L, N, d)
    i = torch.arange(L, device="cuda")[None]
    first = i < (L + 1) // 2 if order == "halves" else i % 2 == 0
    b, e = torch.where(first, 0, z).int(), torch.where(first, a, N).int()
    want = _run(q, k, v, dout, b, e)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").bfloat16()
    k, v = k.clone(), v.clone()
    k[:, :, a:z] = v[:, :, a:z] = bad[torch.arange(d, device="cuda") % 3]
    got = _run(q, k, v, dout, b, e)
    for n in want:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("H,K,L,N,mask", [(2, 2, 300, 300, "causal"), (2, 1, 300, 700, "random"),
                                          (1, 1, 2100, 3500, "window"), (1, 1, 600, 3500, "random")])
def test_keys_reach_only_the_query_gradients_that_see_them(H, K, L, N, mask):
    """NaN in a key: dq is NaN in the rows that see it, and the others keep
    their bits."""
    q, k, v, dout = _inputs(1, H, K, L, N, 64)
    b, e = _ranges(mask, 1, L, N)
    want = _run(q, k, v, dout, b, e)
    j = N - N // 4
    k = k.clone()
    k[:, :, j] = float("nan")
    got = _run(q, k, v, dout, b, e)
    sees = ((b.clamp(0, N) <= j) & (j < e.clamp(0, N)))[0]
    assert sees.any() and not sees.all()
    assert torch.isnan(got["dq"][0][:, sees]).all()
    assert torch.equal(got["dq"][0][:, ~sees], want["dq"][0][:, ~sees])


@pytest.mark.parametrize("H,K,L,N", [(2, 2, 60, 4000), (1, 1, 1, 20000), (1, 1, 4, 60000), (1, 1, 9, 4000)])
def test_nan_survives_the_join_of_split_keys(H, K, L, N):
    """Where the keys of few rows are split: a NaN that is the only key a row
    sees of a part, a whole part of NaN, and a query of NaN."""
    q, k, v, _ = _inputs(1, H, K, L, N, 64)
    for lo, hi, bad in [(0, j + 1, slice(j, j + 1)) for j in range(0, N, 96 if N < 5000 else 1024)] + \
                       [(0, N, slice(N // 2, N)), (5, N, slice(5, N // 2))]:
        b = torch.full((1, L), lo, dtype=torch.int32, device="cuda")
        e = torch.full((1, L), hi, dtype=torch.int32, device="cuda")
        if L > 1:
            e[0, L // 2:] = N                 # the other rows keep the parts where they are
        x = k.clone()
        x[:, :, bad] = float("nan")
        out, lse = ops.httm_attention_forward(q, x, v, b, e)
        assert torch.isnan(out).all() and torch.isnan(lse).all(), (lo, hi, bad)
    q = q.clone()
    q[0, 0, L // 2] = float("nan")
    out, lse = ops.httm_attention_forward(q, k, v)
    rows = torch.arange(L, device="cuda") != L // 2
    assert torch.isnan(out[0, 0, L // 2]).all() and torch.isnan(lse[0, 0, L // 2])
    assert torch.isfinite(out[0, :, rows]).all() and torch.isfinite(lse[0, :, rows]).all()


@pytest.mark.parametrize("N", [3000, 40000])
def test_cleaned_values_leave_later_keys_alone(N):
    """Few rows: infinities and NaN in a channel of the values of every other
    tile of 32 keys, all of which some row does not see; the loads that reuse
    the cleaned tiles' memory bring the keys behind them whole."""
    H, K, L, d = 4, 2, 3, 64
    q, k, v, _ = _inputs(1, H, K, L, N, d)
    b = torch.tensor([[0, N // 2, N - 40]], dtype=torch.int32, device="cuda")
    e = torch.tensor([[N - 1, N, N]], dtype=torch.int32, device="cuda")
    want, lse = ops.httm_attention_forward(q, k, v, b, e)
    v = v.clone()
    j = torch.arange(N, device="cuda")
    odd = (j // 32 % 2 == 0) & (j < N - 40)
    for i, x in enumerate((float("nan"), float("inf"), -float("inf"))):
        v[:, :, odd & (j % 3 == i), 5] = x
    for _ in range(20):
        out, lse2 = ops.httm_attention_forward(q, k, v, b, e)
        rest = torch.arange(d, device="cuda") != 5
        assert torch.equal(lse, lse2) and torch.equal(out[..., rest], want[..., rest])
        assert torch.isnan(out[0, :, :2, 5]).all() and torch.equal(out[0, :, 2, 5], want[0, :, 2, 5])


@pytest.mark.parametrize("B,H,K,L,N", [(16, 1, 1, 1, 8192), (4, 16, 4, 1, 8192), (1, 16, 16, 2, 4000), (1, 2, 2, 60, 4000)])
def test_a_workspace_of_the_extents_serves_calls_with_ranges(B, H, K, L, N):
    q, k, v, dout = _inputs(B, H, K, L, N, 64)
    need_f, need_b = ops.httm_attention_workspace_bytes(B, H, K, L, N, 64)
    guard = 4096
    for b, e in ((None, None), ops.causal_ranges(B, L, N), ops.causal_ranges(B, L, N, window=N // 3)):
        want = _run(q, k, v, dout, b, e)
        ws = torch.full((max(need_f, need_b) + guard,), 0xA5, dtype=torch.uint8, device="cuda")
        out, lse = ops.httm_attention_forward(q, k, v, b, e, workspace=ws[:need_f])
        assert torch.equal(out, want["out"]) and torch.equal(lse, want["lse"]) and (ws[need_f:] == 0xA5).all()
        ws.fill_(0xA5)
        grads = ops.httm_attention_backward(dout, q, k, v, out, lse, b, e, workspace=ws[:need_b])
        assert (ws[need_b:] == 0xA5).all()
        for n, t in zip(("dq", "dk", "dv"), grads):
            assert torch.equal(t, want[n]), n


@pytest.mark.parametrize("G,L,N,mask", [(1, 600, 5000, "random"), (1, 18900, 5000, "random"), (2, 9500, 9000, "random"),
                                        (2, 300, 20000, "random"), (1, 700, 700, "causal"), (4, 5, 9000, "random")])
def test_scattered_infinities_reach_exactly_the_rows_that_see_them(G, L, N, mask):
    """One value in 2,000 an infinity or NaN: a row and channel that sees none
    keeps its bits; else it is what the seen ones add up to."""
    K, d = 2, 64
    q, k, v, _ = _inputs(1, K * G, K, L, N, d)
    b, e = _ranges(mask, 1, L, N)
    want, lse = ops.httm_attention_forward(q, k, v, b, e)
    g = torch.Generator(device="cuda").manual_seed(11)
    kind = torch.randint(0, 6000, v.shape, generator=g, device="cuda")
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").bfloat16()
    v = torch.where(kind < 3, bad[kind.clamp(max=2)], v)
    out, lse2 = ops.httm_attention_forward(q, k, v, b, e)
    assert torch.equal(lse, lse2)
    lo, hi = b.long().clamp(0, N)[0], e.long().clamp(0, N)[0]
    hi = torch.maximum(lo, hi)
    seen = []
    for x in range(3):                        # [kv_heads, L, d]: does the row see one of them?
        n = torch.nn.functional.pad((kind[0] == x).int().cumsum(1), (0, 0, 1, 0))
        seen.append((n[:, hi] - n[:, lo] > 0).repeat_interleave(G, 0))
    nan, pos, neg = seen[0] | seen[1] & seen[2], seen[1], seen[2]
    got = out[0]
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got == float("inf"), pos & ~nan) and torch.equal(got == -float("inf"), neg & ~nan)
    rest = ~(nan | pos | neg)
    assert torch.equal(got[rest], want[0][rest])


def test_a_nan_value_does_not_cost_a_walk_over_all_values():
    """Device time of a causal call with two NaN values against one without
    (walking every key a row sees took 44 times as long, the marked ones 2)."""
    q, k, v, _ = _inputs(1, 1, 1, 4096, 4096, 64)
    b, e = ops.causal_ranges(1, 4096, 4096)
    bad = v.clone()
    bad[:, :, 50] = bad[:, :, 3996] = float("nan")

    def best(x):
        times = []
        for _ in range(10):
            t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            t0.record()
            for _ in range(5):
                ops.httm_attention_forward(q, k, x, b, e)
            t1.record()
            t1.synchronize()
            times.append(t0.elapsed_time(t1))
        return min(times)

    assert best(bad) < 8 * best(v)


@pytest.mark.parametrize("H,K,L,N,d,mask", [(2, 2, 40, 1369, 64, "none"), (16, 4, 64, 1369, 64, "causal"),
                                            (16, 4, 317, 2738, 40, "random"), (3, 1, 200, 8192, 64, "window"),
                                            (2, 1, 130, 5000, 64, "packed"), (6, 2, 34, 1500, 8, "padded")])
def test_split_keys_of_mid_sized_calls(H, K, L, N, d, mask):
    """Up to 8,192 keys and too few query rows to fill the SMs: the keys are
    split among blocks that share an SM, and joined."""
    assert ops.httm_attention_workspace_bytes(1, H, K, L, N, d)[0] > 0
    test_against_definition((1, H, K, L, N, d, mask))


@pytest.mark.parametrize("B,H,K,L,N", [
    (1, 2, 2, 19000, 9000),                    # whole items, more than 8,192 keys
    (1, 1, 1, 300, 200000),                    # split
    (2, 4, 2, 1000, 1400),                     # two blocks an SM
    (16, 16, 16, 1, 41070),                    # few rows, parts added up inside a cluster
    (32, 16, 4, 1, 41070),                     # ... through the workspace
])
def test_waits_that_run_out_set_the_status_and_the_context_recovers(B, H, K, L, N):
    """Failure detection without a fault: with no budget the first waits that
    the hardware does not bridge by itself (some microseconds; the calls are
    long enough) give up, the status says so, the kernels free what they hold
    and exit; with the usual budget the same calls give the same bits as
    before."""
    from token_merging_view_b200 import binding
    q, k, v, dout = _inputs(B, H, K, L, N, 64)
    b, e = ops.causal_ranges(B, L, N)
    want = _run(q, k, v, dout, b, e)
    for call in (lambda: ops.httm_attention_forward(q, k, v, b, e),
                 lambda: ops.httm_attention_backward(dout, q, k, v, want["out"], want["lse"], b, e)):
        try:
            ops.httm_ops_set_wait_budget(0)
            call()
            assert ops.httm_ops_device_status() & binding.HTTM_DEV_TIMEOUT
        finally:
            ops.httm_ops_set_wait_budget(2_000_000_000)
        assert ops.httm_ops_device_status() == 0
        again = _run(q, k, v, dout, b, e)
        for n in want:
            assert torch.equal(again[n], want[n]), n
