"""The operators around one VGGT-style attention block, as cases to time and
check: attention over key ranges (single tokens against a cache, prefill, and
the training step), rotary positions written into the head layout, and the
norms before and after a block fused with its gate and residual.

`run` computes a case either in its plain form (elementary torch operations)
or, with `own` set, through the calls of token_merging_view_b200.  `exact`
gives the same outputs from the definitions in 64 bits.

Sizes are those of the workloads of this repository (37 x 37 = 1369 patch
tokens a frame, 16 heads of 64 channels, 1024 channels a token) and odd ones
around them.
"""
import math

import torch

own = False

PATCHES = 1369  # tokens of one frame: a 37 x 37 patch grid
EPS = 1e-5


# ------------------------------------------------------------------ cases
def attention(name, **kw):
    base = dict(op="attention", batch=1, heads=16, kv_heads=16, q_len=1, kv_len=PATCHES, d=64, mask="none",
                window=0, frame=PATCHES, train=False)
    return {**({"name": name} if name else {}), **base, **kw}


def rotary(name, **kw):
    base = dict(op="rotary", batch=1, tokens=1, heads=16, kv_heads=16, d=64, rotary_dim=64, axes=1, layout="half",
                dtype="bf16", base=10000.0, scaling="none", scale=1.0, far=0, train=False)
    return {**({"name": name} if name else {}), **base, **kw}


def norm(name, **kw):
    base = dict(op="norm", rows=PATCHES, ch=1024, stream="bf16", branch="bf16", pre="layer", post="none",
                gates=1, residual_scale=1.0, train=False)
    return {**({"name": name} if name else {}), **base, **kw}


def listed():
    return [
        # the smallest serving call: one new token of one sequence against the cache of one frame
        attention("decode_one"),
        # a serving step of 32 sequences with ragged caches of up to 30 frames, four query heads to a key head
        attention("decode_ragged", batch=32, kv_heads=4, kv_len=30 * PATCHES, mask="padded"),
        # a new frame of a stream attends to itself and the nine frames before it
        attention("prefill_frame", q_len=PATCHES, kv_len=10 * PATCHES, mask="frames"),
        # a small fine-tuning step with an odd length, narrow heads shared by three, and a sliding window
        attention("train_window", batch=3, heads=6, kv_heads=2, q_len=317, kv_len=317, d=40, mask="window",
                  window=100, train=True),
        # frame attention of 8 images whose patch counts differ (a padded batch): forward and gradients
        attention("train_padded", batch=8, q_len=PATCHES, kv_len=PATCHES, mask="padded", train=True),
        # global attention over 8 frames, every token to every token: forward and gradients
        attention("train_global", q_len=8 * PATCHES, kv_len=8 * PATCHES, train=True),
        # the residual update and next norm of one image
        norm("norm_frame"),
        # the same of 30 frames with its backward pass
        norm("norm_train", rows=30 * PATCHES, train=True),
        # a norm on both sides of the block, fp32 residual stream, a gate for each of 4 frames, odd width
        norm("norm_train_both", rows=4 * PATCHES, ch=1001, stream="f32", pre="rms", post="rms", gates=4,
             residual_scale=0.7, train=True),
        # queries and keys of 30 frames turned by their grid row and column, and the way back of their gradients
        rotary("rotary_grid", tokens=30 * PATCHES, axes=2, base=100.0, train=True),
        # one token each of 32 sequences far along, a part of the head, adjacent pairs, stretched frequencies
        rotary("rotary_decode", batch=32, kv_heads=4, rotary_dim=32, layout="pairs", scaling="yarn", scale=16.0,
               far=500000),
        # fp32 heads of an odd size over one sequence, linearly interpolated positions
        rotary("rotary_f32", batch=2, tokens=2003, heads=5, kv_heads=1, d=50, rotary_dim=26, dtype="f32",
               scaling="linear", scale=4.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["decode", "prefill", "train", "train", "norm", "norm", "rotary"])
    if kind == "decode":
        group = rng.choice([1, 2, 3, 4, 8])
        kv_heads = rng.choice([1, 2, 4, 5, 8])
        return attention(None, batch=_log(rng, 1, 48), heads=kv_heads * group, kv_heads=kv_heads,
                         q_len=rng.choice([1, 1, 1, 2, 5]), kv_len=_log(rng, 30, 30 * PATCHES),
                         d=rng.choice([64, 64, 48, 32]), mask=rng.choice(["none", "padded", "causal"]))
    if kind == "prefill":
        n = _log(rng, 100, 4 * PATCHES)
        return attention(None, q_len=n, kv_len=n + _log(rng, 1, 6 * PATCHES), kv_heads=rng.choice([1, 4, 16]),
                         d=rng.choice([64, 56]), mask=rng.choice(["frames", "causal", "window", "none"]),
                         window=_log(rng, 1, 2000), frame=_log(rng, 50, 1500))
    if kind == "train":
        n, kv_heads = _log(rng, 17, 5 * PATCHES), rng.choice([1, 2, 4])
        most = max(1, min(16, int(4e8 / (n * n * 4 * kv_heads))))
        return attention(None, batch=_log(rng, 1, most), heads=kv_heads * rng.choice([1, 2, 4]), kv_heads=kv_heads,
                         q_len=n, kv_len=n, d=rng.choice([64, 64, 40, 16, 8]),
                         mask=rng.choice(["none", "padded", "causal", "window", "frames"]),
                         window=_log(rng, 1, 1000), frame=_log(rng, 20, 1500), train=True)
    if kind == "norm":
        gates = rng.choice([0, 1, 1, 3, 8])
        stream, branch = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
        return norm(None, rows=max(1, gates) * _log(rng, 1, 12 * PATCHES // max(1, gates)), ch=_log(rng, 24, 2500),
                    stream=stream, branch=branch, pre=rng.choice(["layer", "rms", "none"]),
                    post=rng.choice(["none", "none", "layer", "rms"]), gates=gates,
                    residual_scale=rng.choice([1.0, 1.0, 0.5]), train=rng.random() < 0.7)
    axes = rng.choice([1, 1, 2])
    d = rng.choice([16, 40, 64, 64, 50, 128])
    rot = rng.choice([d, d // 2]) // (2 * axes) * (2 * axes)
    kv_heads = rng.choice([1, 2, 8])
    return rotary(None, batch=rng.choice([1, 1, 2, 16]), tokens=_log(rng, 1, 4000), heads=kv_heads * rng.choice([1, 2, 3]),
                  kv_heads=kv_heads, d=d, rotary_dim=rot, axes=axes, layout=rng.choice(["half", "pairs"]),
                  dtype=rng.choice(["bf16", "bf16", "f32"]), base=rng.choice([100.0, 10000.0, 500000.0]),
                  scaling=rng.choice(["none", "linear", "yarn"]), scale=rng.choice([2.0, 8.0, 32.0]),
                  far=rng.choice([0, 0, 100000, 1000000]), train=rng.random() < 0.4)


DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def key_ranges(c):
    """Each query's keys [begin, end) as int32 [batch, q_len] on the CPU, or (None, None)."""
    if c["mask"] == "none":
        return None, None
    at = torch.arange(c["q_len"]) + (c["kv_len"] - c["q_len"])  # the queries are the last tokens of the keys
    if c["mask"] == "padded":
        length = torch.tensor([c["kv_len"] - b * 613 % (c["kv_len"] * 3 // 4 + 1) for b in range(c["batch"])])
        live = (at[None] < length[:, None]) | (c["q_len"] < c["kv_len"])
        end = torch.where(live, length[:, None], 0)
        return torch.zeros_like(end).int(), end.int()
    end = at + 1
    if c["mask"] == "frames":
        end = torch.clamp((at // c["frame"] + 1) * c["frame"], max=c["kv_len"])
    begin = torch.clamp(at + 1 - c["window"], min=0) if c["mask"] == "window" else torch.zeros_like(end)
    rows = (c["batch"], c["q_len"])
    return begin.expand(rows).contiguous().int(), end.expand(rows).contiguous().int()


def frequencies(c):
    """float64 radians a position for each pair of one axis, and the factor on cosine and sine."""
    n = c["rotary_dim"] // (2 * c["axes"])
    f = c["base"] ** (-torch.arange(n, dtype=torch.float64) / n)
    s = c["scale"]
    if c["scaling"] == "linear":
        return f / s, 1.0
    if c["scaling"] == "yarn":
        # pairs that turn less than once in the first 4096 positions are interpolated, those of over 32 turns kept
        turns = 4096 * f / (2 * math.pi)
        keep = torch.clamp((turns - 1) / (32 - 1), 0, 1)
        return f * keep + f / s * (1 - keep), 0.1 * math.log(s) + 1.0
    return f, 1.0


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape, dtype=torch.bfloat16, scale=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale + mean).to(dtype)

    st = {"case": c}
    if c["op"] == "attention":
        b, e = key_ranges(c)
        st["begin"], st["end"] = (None, None) if b is None else (b.cuda(), e.cuda())
        st["q"] = rand(c["batch"], c["heads"], c["q_len"], c["d"])
        st["k"] = rand(c["batch"], c["kv_heads"], c["kv_len"], c["d"])
        # values stay where the projection left them: tokens outermost, then heads
        st["v"] = rand(c["batch"], c["kv_len"], c["kv_heads"], c["d"]).transpose(1, 2)
        if c["train"]:
            st["dout"] = rand(c["batch"], c["heads"], c["q_len"], c["d"])
    elif c["op"] == "rotary":
        dt = DTYPE[c["dtype"]]
        h, hk, d = c["heads"], c["kv_heads"], c["d"]
        packed = rand(c["batch"], c["tokens"], h + 2 * hk, d, dtype=dt)  # the projection's output
        st["q"], st["k"] = packed[:, :, :h].transpose(1, 2), packed[:, :, h:h + hk].transpose(1, 2)
        if c["axes"] == 2:  # grid rows and columns of 37 x 37 patches
            n = torch.arange(c["tokens"], device="cuda") % PATCHES
            pos = torch.stack([n // 37, n % 37], -1).expand(c["batch"], -1, -1)
        else:
            start = torch.randint(0, c["far"] + 1, (c["batch"], 1, 1), generator=g, device="cuda")
            pos = start + torch.arange(c["tokens"], device="cuda")[None, :, None]
        st["pos"] = pos.contiguous().int()
        f, st["factor"] = frequencies(c)
        st["freqs"] = f.cuda()
        if c["train"]:
            st["dq"] = rand(c["batch"], h, c["tokens"], d, dtype=dt)
            st["dk"] = rand(c["batch"], hk, c["tokens"], d, dtype=dt)
    else:
        n, ch, f32 = c["rows"], c["ch"], torch.float32
        st["x"] = rand(n, ch, dtype=DTYPE[c["stream"]], scale=2.0, mean=0.3)
        st["f"] = rand(n, ch, dtype=DTYPE[c["branch"]], mean=0.1)
        st["gate"] = rand(c["gates"], ch, dtype=f32, scale=0.5) if c["gates"] else None
        for side in ("post", "pre"):
            layer = c[side] == "layer"
            st[side] = None if c[side] == "none" else (rand(ch, dtype=f32, scale=0.2, mean=1.0),
                                                       rand(ch, dtype=f32, scale=0.2) if layer else None)
        if c["train"]:
            st["dy"] = rand(n, ch, dtype=DTYPE[c["stream"]])
            st["dz"] = rand(n, ch, dtype=DTYPE[c["branch"]]) if c["pre"] != "none" else None
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"attention": own_attention, "rotary": own_rotary, "norm": own_norm}[op](state)
    return {"attention": plain_attention, "rotary": plain_rotary, "norm": plain_norm}[op](state)


def plain_attention(st):
    c = st["case"]
    B, H, L, D = st["q"].shape
    G, K, N = H // st["k"].shape[1], st["k"].shape[1], st["k"].shape[2]
    scale = D ** -0.5
    q, k, v = st["q"].float().reshape(B, K, G * L, D), st["k"].float(), st["v"].float()
    s = (q @ k.transpose(2, 3)) * scale
    if st["begin"] is not None:
        j = torch.arange(N, device=s.device)
        seen = (j >= st["begin"][..., None]) & (j < st["end"][..., None])  # [B, L, N]
        s = s.view(B, K, G, L, N).masked_fill(~seen[:, None, None], -math.inf).view(B, K, G * L, N)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    p = torch.exp(s - m)
    del s
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    out = p @ v
    res = {"out": out.view(B, H, L, D).to(torch.bfloat16), "lse": (m + torch.log(total)).view(B, H, L)}
    if c["train"]:
        do = st["dout"].float().reshape(B, K, G * L, D)
        dp = do @ v.transpose(2, 3)
        ds = p * (dp - (do * out).sum(-1, keepdim=True)) * scale
        res["dq"] = (ds @ k).view(B, H, L, D).to(torch.bfloat16)
        res["dk"] = (ds.transpose(2, 3) @ q).to(torch.bfloat16)
        res["dv"] = (p.transpose(2, 3) @ do).to(torch.bfloat16)
    return res


def plain_turn(x, cos, sin, c):
    """x [batch, heads, tokens, d] in fp32; cos, sin [batch, 1, tokens, axes, pairs]."""
    r, pairs = c["rotary_dim"], c["rotary_dim"] // (2 * c["axes"])
    part = x[..., :r].unflatten(-1, (c["axes"], 2, pairs) if c["layout"] == "half" else (c["axes"], pairs, 2))
    a, b = part.unbind(-2 if c["layout"] == "half" else -1)
    turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -2 if c["layout"] == "half" else -1)
    return torch.cat([turned.flatten(-3), x[..., r:]], -1)


def plain_rotary(st):
    c = st["case"]
    angle = (st["pos"].double()[..., None] * st["freqs"])[:, None]  # far positions need the 64 bits
    cos, sin = (torch.cos(angle) * st["factor"]).float(), (torch.sin(angle) * st["factor"]).float()
    dt = st["q"].dtype
    res = {"q": plain_turn(st["q"].float(), cos, sin, c).to(dt), "k": plain_turn(st["k"].float(), cos, sin, c).to(dt)}
    if c["train"]:
        res["dq"] = plain_turn(st["dq"].float(), cos, -sin, c).to(dt)
        res["dk"] = plain_turn(st["dk"].float(), cos, -sin, c).to(dt)
    return res


def plain_normed(x, kind):
    """(x normalised without weight and bias, 1 / deviation)."""
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def plain_normed_grad(g, hat, r, kind):
    g = g - hat * (g * hat).mean(-1, keepdim=True) - (g.mean(-1, keepdim=True) if kind == "layer" else 0.0)
    return g * r


def plain_norm(st):
    c = st["case"]
    x, f = st["x"].float(), st["f"].float()
    a, gate = f, 1.0
    if st["gate"] is not None:
        gate = st["gate"].repeat_interleave(c["rows"] // c["gates"], 0)
    if st["post"]:
        fhat, fr = plain_normed(f, c["post"])
        a = fhat * st["post"][0] + (st["post"][1] if st["post"][1] is not None else 0.0)
    y = (c["residual_scale"] * x + gate * a).to(DTYPE[c["stream"]])
    res = {"y": y}
    if st["pre"]:
        hat, r = plain_normed(y.float(), c["pre"])  # the norm reads the stream as it is stored
        z = hat * st["pre"][0] + (st["pre"][1] if st["pre"][1] is not None else 0.0)
        res["z"] = z.to(DTYPE[c["branch"]])
    if c["train"]:
        g = st["dy"].float()
        if st["pre"]:
            dz = st["dz"].float()
            g = g + plain_normed_grad(dz * st["pre"][0], hat, r, c["pre"])
            res["dpre_weight"] = (dz * hat).sum(0)
            if st["pre"][1] is not None:
                res["dpre_bias"] = dz.sum(0)
        res["dx"] = (c["residual_scale"] * g).to(DTYPE[c["stream"]])
        if st["gate"] is not None:
            res["dgate"] = (g * a).view(c["gates"], -1, c["ch"]).sum(1)
        df = g * gate
        if st["post"]:
            res["dpost_weight"] = (df * fhat).sum(0)
            if st["post"][1] is not None:
                res["dpost_bias"] = df.sum(0)
            df = plain_normed_grad(df * st["post"][0], fhat, fr, c["post"])
        res["df"] = df.to(DTYPE[c["branch"]])
    return res


# ------------------------------------------------------------------ the framework's calls
def own_attention(st):
    from token_merging_view_b200 import ops
    mask = dict(key_begin=st["begin"], key_end=st["end"])
    out, lse = ops.httm_attention_forward(st["q"], st["k"], st["v"], **mask)
    res = {"out": out, "lse": lse}
    if st["case"]["train"]:
        res["dq"], res["dk"], res["dv"] = ops.httm_attention_backward(st["dout"], st["q"], st["k"], st["v"], out, lse,
                                                                      **mask)
    return res


def own_rotary(st):
    from token_merging_view_b200 import ops
    c = st["case"]
    layout = ops.HTTM_ROTARY_HALF if c["layout"] == "half" else ops.HTTM_ROTARY_PAIRS
    how = dict(axes=c["axes"], layout=layout, factor=st["factor"])
    res = {}
    res["q"], res["k"] = ops.httm_rotary(st["q"], st["k"], st["freqs"], st["pos"], **how)
    if c["train"]:
        res["dq"], res["dk"] = ops.httm_rotary(st["dq"], st["dk"], st["freqs"], st["pos"], inverse=True, **how)
    return res


def own_norm(st):
    from token_merging_view_b200 import ops
    c = st["case"]
    kind = {"layer": ops.HTTM_NORM_LAYER, "rms": ops.HTTM_NORM_RMS}
    how = {side: ops.Norm(kind[c[side]], *st[side], eps=EPS) for side in ("post", "pre") if st[side]}
    how.update(gate=st["gate"], residual_scale=c["residual_scale"])
    y, z, stats = ops.httm_gated_norm_forward(st["x"], st["f"], **how)
    res = {"y": y}
    if st["pre"]:
        res["z"] = z
    if c["train"]:
        grads = ops.httm_gated_norm_backward(st["dy"], st["dz"], st["f"], y, stats, **how)
        res.update({k: t for k, t in grads.items() if t is not None})
    return res


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "attention":
        B, H, K, L, N, D = (c[k] for k in ("batch", "heads", "kv_heads", "q_len", "kv_len", "d"))
        b, e = key_ranges(c)
        if b is None:
            pairs, keys = B * L * N, B * N
        else:
            pairs = int((e.long() - b.long()).clamp(min=0).sum())
            keys = int((e.amax(1).long() - torch.where(e > b, b, N).amin(1).long()).clamp(min=0).sum())
        rows = B * H * L
        moved = rows * D * 2 * 2 + rows * 4 + keys * K * D * 2 * 2
        flops = 4 * D * pairs * H
        if c["train"]:  # q, k, v, out, lse and dout read, dq, dk, dv written; five products of the same size
            moved += rows * D * 2 * 4 + rows * 4 + keys * K * D * 2 * 2 + B * N * K * D * 2 * 2
            flops += 10 * D * pairs * H
        return {"bytes": moved, "flops": flops}
    if c["op"] == "rotary":
        es, times = (2 if c["dtype"] == "bf16" else 4), (2 if c["train"] else 1)
        rows = c["batch"] * c["tokens"] * (c["heads"] + c["kv_heads"])
        return {"bytes": times * (2 * rows * c["d"] * es + c["batch"] * c["tokens"] * c["axes"] * 4),
                "flops": times * rows * c["rotary_dim"] * 3}
    xs, fs = (2 if c[k] == "bf16" else 4 for k in ("stream", "branch"))
    n, pre = c["rows"] * c["ch"], c["pre"] != "none"
    moved, flops = n * (2 * xs + fs * (2 if pre else 1)), n * 20
    if c["train"]:  # dy, dz, f and y read, dx and df written
        moved += n * (2 * xs + 2 * fs + (xs + fs if pre else 0))
        flops += n * 40
    return {"bytes": moved, "flops": flops}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"attention": exact_attention, "rotary": exact_rotary, "norm": exact_norm}[case["op"]](case, st)


def exact_attention(c, st):
    B, H, L, D = st["q"].shape
    K, N = st["k"].shape[1], st["k"].shape[2]
    new = lambda like: torch.zeros(like.shape, dtype=torch.float64, device="cuda")  # noqa: E731
    res = {"out": new(st["q"]), "lse": new(st["q"][..., 0])}
    if c["train"]:
        res.update(dq=new(st["q"]), dk=new(st["k"]), dv=new(st["v"]))
    keys = torch.arange(N, device="cuda")
    for b in range(B):
        hidden = None
        if st["begin"] is not None:
            hidden = (keys[None] < st["begin"][b][:, None]) | (keys[None] >= st["end"][b][:, None])
        for h in range(H):
            n = h * K // H
            q, k, v = st["q"][b, h].double(), st["k"][b, n].double(), st["v"][b, n].double()
            score = q @ k.T / math.sqrt(D)
            if hidden is not None:
                score[hidden] = -math.inf
            lse = torch.logsumexp(score, 1)
            prob = torch.nan_to_num(torch.exp(score - lse[:, None]), nan=0.0)
            res["lse"][b, h], res["out"][b, h] = lse, prob @ v
            if c["train"]:
                g = st["dout"][b, h].double()
                res["dv"][b, n] += prob.T @ g
                inner = g @ v.T
                inner = prob * (inner - (prob * inner).sum(1, keepdim=True)) / math.sqrt(D)
                res["dq"][b, h] = inner @ k
                res["dk"][b, n] += inner.T @ q
    return res


def exact_rotary(c, st):
    pairs, r = c["rotary_dim"] // (2 * c["axes"]), c["rotary_dim"]
    # which channels pair up, and the axis and frequency of each pair
    i = torch.arange(r // 2, device="cuda")
    axis, n = i // pairs, i % pairs
    lo = axis * 2 * pairs + n if c["layout"] == "half" else 2 * i
    hi = lo + (pairs if c["layout"] == "half" else 1)
    theta = st["pos"].double()[..., axis] * st["freqs"][n]  # [batch, tokens, pairs of all axes]
    turn = st["factor"] * torch.polar(torch.ones_like(theta), theta)[:, None]

    def turned(x, t):
        x = x.double()
        z = torch.complex(x[..., lo], x[..., hi]) * t
        x[..., lo], x[..., hi] = z.real, z.imag
        return x

    res = {"q": turned(st["q"], turn), "k": turned(st["k"], turn)}
    if c["train"]:
        res.update(dq=turned(st["dq"], turn.conj()), dk=turned(st["dk"], turn.conj()))
    return res


def exact_norm(c, st):
    def normal(v, kind, weight, bias):
        if kind == "layer":
            v = v - v.mean(1, keepdim=True)
        v = v / torch.sqrt((v ** 2).mean(1, keepdim=True) + EPS) * weight.double()
        return v if bias is None else v + bias.double()

    def leaf(t):
        return None if t is None else t.double().requires_grad_(c["train"])

    x, f, gate = leaf(st["x"]), leaf(st["f"]), leaf(st["gate"])
    post = [leaf(t) for t in st["post"]] if st["post"] else [None, None]
    pre = [leaf(t) for t in st["pre"]] if st["pre"] else [None, None]
    a = f if post[0] is None else normal(f, c["post"], *post)
    if gate is not None:
        a = (a.view(c["gates"], -1, c["ch"]) * gate[:, None]).view_as(a)
    y = c["residual_scale"] * x + a
    y = y + (y.to(DTYPE[c["stream"]]).double() - y).detach()  # as the stream stores it
    res, z = {"y": y.detach()}, None
    if pre[0] is not None:
        z = normal(y, c["pre"], *pre)
        res["z"] = z.detach()
    if c["train"]:
        loss = (y * st["dy"].double()).sum()
        if z is not None:
            loss = loss + (z * st["dz"].double()).sum()
        wanted = {"dx": x, "df": f, "dgate": gate, "dpre_weight": pre[0], "dpre_bias": pre[1],
                  "dpost_weight": post[0], "dpost_bias": post[1]}
        wanted = {k: t for k, t in wanted.items() if t is not None}
        res.update(zip(wanted, torch.autograd.grad(loss, list(wanted.values()))))
    return res
