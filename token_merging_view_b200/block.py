"""The attention half of a VGGT-style block on one GPU, serving and training.

    z  = norm1(x)                               (or handed in by the block before)
    q, k, v = heads of z @ qkv_weight^T
    q, k    = turned by the patch's grid row and column
    o  = attention(q, k, v)                     merged (a plan), or over key ranges
    y  = x + gate * (o @ proj_weight^T)         and  z' = norm2(y)

Everything but the two library matrix products runs in this package's
kernels: :func:`httm_gated_norm_forward` joins the residual, the gate
(LayerScale) and the next norm in one pass, :func:`httm_rotary` reads the
packed projection and writes the [h, N, d] layout that
:func:`httm_forward` and :func:`httm_attention_forward` take.  The merged
layer ("HTTM: Head-wise Temporal Token Merging for Faster VGGT", overall
framework) is for serving; gradients go through attention over key ranges.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from .binding import httm_forward
from .ops import (Norm, httm_attention_backward, httm_attention_forward, httm_gated_norm_backward,
                  httm_gated_norm_forward, httm_rotary)


def grid_positions(T: int, grid: int, device="cuda") -> torch.Tensor:
    """int32 [T * grid * grid, 2]: each token's patch row and column."""
    p = torch.arange(T * grid * grid, device=device) % (grid * grid)
    return torch.stack([torch.div(p, grid, rounding_mode="floor"), p % grid], -1).int()


@dataclass
class GlobalAttentionBlock:
    """heads; qkv_weight [3 C, C] and proj_weight [C, C] in bfloat16; gate
    float32 [C]; norm1 (of x) and norm2 (of the new stream); freqs float64
    [d / 4] (the turn of each channel pair of a row or column half)."""
    heads: int
    qkv_weight: torch.Tensor
    proj_weight: torch.Tensor
    gate: torch.Tensor
    norm1: Norm
    norm2: Norm
    freqs: torch.Tensor

    def _heads(self, z, positions):
        """q, k turned and v as it lies, each [heads, N, d]."""
        N, C = z.shape
        packed = (z @ self.qkv_weight.t()).view(N, 3, self.heads, C // self.heads)
        q, k, v = (packed[:, i].transpose(0, 1) for i in range(3))
        q, k = httm_rotary(q, k, self.freqs, positions, axes=2)
        return q, k, v

    def forward(self, x, positions, z=None, plan=None, workspace=None, key_begin=None, key_end=None):
        """(y, z', saved) for the stream x [N, C] (positions int32 [N, 2]).

        z: norm1(x) if the block before has it already (then ``backward``
        returns its gradient as dz).  plan: a merge plan of N tokens -- the
        layer runs merged, and saved is None.  key_begin, key_end: int32 [N]
        key ranges (with a plan: not supported)."""
        stats1 = None
        given = z is not None
        if not given:
            _, z, stats1 = httm_gated_norm_forward(x, pre=self.norm1, branch_dtype=self.qkv_weight.dtype)
        q, k, v = self._heads(z, positions)
        if plan is not None:
            if key_begin is not None or key_end is not None:
                raise ValueError("a merge plan takes no key ranges")
            o, lse = httm_forward(plan, q, k, v.contiguous(), workspace=workspace), None
        else:
            o, lse = httm_attention_forward(q, k, v, key_begin, key_end)
        a = o.transpose(0, 1).reshape(x.shape)
        f = a @ self.proj_weight.t()
        y, z_next, stats2 = httm_gated_norm_forward(x, f, gate=self.gate, pre=self.norm2)
        saved = None if plan is not None else dict(
            x=x, z=z, given=given, stats1=stats1, q=q, k=k, v=v, o=o, lse=lse, a=a, f=f, y=y, stats2=stats2,
            positions=positions, key_begin=key_begin, key_end=key_end)
        return y, z_next, saved

    def backward(self, dy, dz_next, saved):
        """Gradients of sum(dy * y) + sum(dz_next * z'): a dict of dx (and dz,
        if z was handed in), dqkv_weight, dproj_weight, dgate and the norms'
        parameters (dnorm1_weight, ...; None where there is none)."""
        if saved is None:
            raise ValueError("the merged layer has no gradient: run forward without a plan")
        s = saved
        g2 = httm_gated_norm_backward(dy, dz_next, s["f"], s["y"], s["stats2"], gate=self.gate, pre=self.norm2)
        df = g2["df"]
        dproj = df.t() @ s["a"]
        N, C = df.shape
        do = (df @ self.proj_weight).view(N, self.heads, C // self.heads).transpose(0, 1)
        # the three gradients land in the packed layout of the projection
        packed = torch.empty(N, 3, self.heads, C // self.heads, dtype=do.dtype, device=do.device)
        dq, dk, dv = (packed[:, i].transpose(0, 1) for i in range(3))
        httm_attention_backward(do, s["q"], s["k"], s["v"], s["o"], s["lse"], s["key_begin"], s["key_end"], dq=dq,
                                dk=dk, dv=dv)
        httm_rotary(dq, dk, self.freqs, s["positions"], axes=2, inverse=True, q_out=dq, k_out=dk)
        dpacked = packed.view(N, 3 * C)
        dqkv = dpacked.t() @ s["z"]
        dz = dpacked @ self.qkv_weight
        out = dict(dqkv_weight=dqkv, dproj_weight=dproj, dgate=g2["dgate"], dnorm2_weight=g2["dpre_weight"],
                   dnorm2_bias=g2["dpre_bias"], dnorm1_weight=None, dnorm1_bias=None)
        if s["given"]:
            return dict(out, dx=g2["dx"], dz=dz)
        g1 = httm_gated_norm_backward(g2["dx"], dz, None, s["x"], s["stats1"], pre=self.norm1)
        return dict(out, dx=g1["dx"], dnorm1_weight=g1["dpre_weight"], dnorm1_bias=g1["dpre_bias"])
