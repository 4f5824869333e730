"""References for the operators around the layer, in 64 bits, with bounds on
what the kernels may be off by.

U is half a step of bf16 relative to the value (2^-8), the most one rounding
can move it.  The fp32 work between roundings is bounded through the number
of additions in a chain: a sum of n terms carries at most n 2^-24 of the sum
of their magnitudes."""
from __future__ import annotations

import math

import torch

U = torch.finfo(torch.bfloat16).eps / 2
# 64 products into a score or a gradient of one (fp32 accumulation in a
# tensor core, which may truncate: twice the rounding), the exponent's
# scaling and the exp unit's own 2^-22: below 2^-15 of the magnitudes
F = 2.0 ** -15


def attention(q, k, v, begin=None, end=None, dout=None, scale=None):
    """out, lse (and dq, dk, dv) of [B, H, L, d] tensors in 64 bits, and the
    most the kernels' results may differ from them, element by element.

    P is rounded to bf16 before P V: U sum_j P |v|; the result is rounded: U
    |out|.  A score is off by at most e_s = F scale sum |q k| + F, which moves P
    by that factor.  D = dout . out takes the rounded out: off by |dout| .
    (bound of out) =: e_D, and dS = P (dP - D) is rounded: U |dS|, and moved by
    P (e_D + F sum |dout v|) and by e_s |dS|."""
    q, k, v = (t.double() for t in (q, k, v))
    B, H, L, d = q.shape
    K, N = k.shape[1], k.shape[2]
    G = H // K
    scale = scale or 1.0 / math.sqrt(d)
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    j = torch.arange(N, device=q.device)
    lo = torch.zeros((B, L), dtype=torch.int64, device=q.device) if begin is None else begin.long().clamp(min=0)
    hi = torch.full((B, L), N, device=q.device) if end is None else end.long().clamp(max=N)
    seen = ((j >= lo[..., None]) & (j < hi[..., None]))[:, None]          # [B, 1, L, N]
    some = seen.any(-1, keepdim=True)
    # what lies outside every range may be anything
    kk = torch.where(seen.any(2)[..., None], kk, 0.0)
    vv = torch.where(seen.any(2)[..., None], vv, 0.0)
    q = torch.where(some, q, 0.0)
    s = (q @ kk.transpose(2, 3) * scale).masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1) if N > 0 else torch.full((B, H, L), -math.inf, dtype=torch.float64, device=q.device)
    P = torch.where(seen, torch.exp(s - torch.where(some, lse[..., None], 0.0)), 0.0)
    e_s = F * scale * (q.abs() @ kk.abs().transpose(2, 3)) + F
    e_s = torch.where(seen, e_s, 0.0)
    e_row = e_s.amax(-1, keepdim=True) if N > 0 else torch.zeros((B, H, L, 1), dtype=torch.float64, device=q.device)
    out = P @ vv
    A = P @ vv.abs()
    tol = {"out": U * (A * (1 + U) + out.abs()) + 2 * e_row * A, "lse": 2 * e_row[..., 0] + 2.0 ** -22 * lse.abs()}
    res = {"out": out, "lse": lse}
    if dout is not None:
        g = torch.where(some, dout.double(), 0.0)
        dP = g @ vv.transpose(2, 3)
        D = (P * dP).sum(-1, keepdim=True)
        dS = P * (dP - D)
        e_D = (g.abs() * tol["out"]).sum(-1, keepdim=True) + F * (g.abs() * out.abs()).sum(-1, keepdim=True)
        e_dS = U * dS.abs() + P * (e_D + F * (g.abs() @ vv.abs().transpose(2, 3))) + 2 * e_row * (1 + U) * dS.abs()
        heads = lambda t: t.view(B, K, G, N, d).sum(2)  # noqa: E731
        res["dq"] = scale * dS @ kk
        tol["dq"] = scale * e_dS @ kk.abs() + (U + F) * res["dq"].abs() + F * scale * dS.abs() @ kk.abs()
        res["dk"] = heads(scale * dS.transpose(2, 3) @ q)
        tol["dk"] = heads(scale * (e_dS + F * dS.abs()).transpose(2, 3) @ q.abs()) + (U + F) * res["dk"].abs()
        res["dv"] = heads(P.transpose(2, 3) @ g)
        e_P = P * (U + 2 * e_row * (1 + U) + F)
        tol["dv"] = heads(e_P.transpose(2, 3) @ g.abs()) + (U + F) * res["dv"].abs()
    return res, tol


def check(got, want, tol, name):
    got, tol = got.double(), tol + 1e-30
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got) & (got == want), inf), f"{name}: infinities"
    err = torch.where(inf, 0.0, (got - want).abs())
    assert torch.isfinite(err).all(), f"{name}: not finite"
    worst = float((err / torch.where(inf, 1.0, tol)).max()) if err.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.2f} times the bound, max error {float(err.max()):.3g}"


# ------------------------------------------------------------------ rotary
def rotary(x, freqs, pos, axes, half, factor, inverse=False):
    """x [B, heads, T, d], pos [B, T, axes]; in 64 bits."""
    pairs = freqs.numel()
    x = x.double().clone()
    for a in range(axes):
        ang = pos[..., a].double()[..., None] * freqs * (-1 if inverse else 1)     # [B, T, pairs]
        c, s = factor * torch.cos(ang)[:, None], factor * torch.sin(ang)[:, None]
        at = a * 2 * pairs
        lo = slice(at, at + pairs) if half else slice(at, at + 2 * pairs, 2)
        hi = slice(at + pairs, at + 2 * pairs) if half else slice(at + 1, at + 2 * pairs, 2)
        u, v = x[..., lo].clone(), x[..., hi].clone()
        x[..., lo], x[..., hi] = u * c - v * s, v * c + u * s
    return x


def rotary_tol(x, freqs, pos, axes, half, factor, dtype):
    """Each output is a sum of two products; cos and sin are within 2^-21
    (fp32 angle in half turns: 2^-25 of one, times pi, the function's own 2
    steps, the factor's rounding) of the frequency as given, plus the fp64
    rounding of frequency and product, 2^-51 of position * frequency."""
    pairs = freqs.numel()
    mag = torch.zeros_like(x, dtype=torch.float64)
    a = x.double().abs()
    for ax in range(axes):
        at = ax * 2 * pairs
        lo = slice(at, at + pairs) if half else slice(at, at + 2 * pairs, 2)
        hi = slice(at + pairs, at + 2 * pairs) if half else slice(at + 1, at + 2 * pairs, 2)
        e = 2.0 ** -21 + (pos[..., ax].double().abs()[..., None] * freqs.abs() * 2.0 ** -51)[:, None]
        m = abs(factor) * (a[..., lo] + a[..., hi]) * e
        mag[..., lo], mag[..., hi] = m, m
    return mag, (U if dtype == torch.bfloat16 else 2.0 ** -24)


# ------------------------------------------------------------------ gated norm
FN = 2.0 ** -17     # fp32 chains of fewer than 128 additions


def normal(v, kind, eps):
    """(n = (v - mean) r, r, bound of n) in 64 bits; kind 1 layer, 2 rms."""
    av = v.abs().mean(1, keepdim=True)
    c = v - v.mean(1, keepdim=True) if kind == 1 else v
    r = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    n = c * r
    # the mean is off by FN mean|v|, the variance by FN of itself plus what the mean's error adds
    return n, r, FN * (2 * n.abs() + r * (v.abs() + av) * (1 + n.abs()))


def normal_grad(g, n, r, e_n, kind):
    """(gradient of v, its bound) for the gradient g of n, with g off by FN |g|."""
    C = g.shape[1]
    m0 = g.mean(1, keepdim=True) if kind == 1 else 0.0
    m1 = (g * n).mean(1, keepdim=True)
    a0, a1 = g.abs().mean(1, keepdim=True), (g.abs() * (n.abs() + e_n / FN)).mean(1, keepdim=True)
    dv = r * (g - m0 - n * m1)
    # r itself is off by FN (1 + r mean|v| ...), part of e_n / FN relative to n
    rel = (e_n / FN / n.abs().clamp(min=1e-3)).amin(1, keepdim=True).clamp(min=2.0)
    e = FN * r * (g.abs() + a0 + (n.abs() + e_n / FN) * a1) * (2 + rel)
    assert C > 0
    return dv, e
