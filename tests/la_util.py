"""64-bit restatements of the decayed linear attention, the query/key preparation and the
pool moves, from their formulas, and random inputs for them (CPU tensors)."""
from __future__ import annotations

import torch

# Relative L2 tolerances.
#  o, bf16     storage, scores and the copy of the state that meets the queries are each
#              rounded once to 8 bits (2^-9 of the value in the mean): 3 * 2^-9
#  o, f32 and states, both types: sums of fp32 products whose factors carry at most 2^-17
#              each (a decay weight; in bf16 storage the weighted key, held as a sum of two
#              bf16): 2 * 2^-17 plus fp32 accumulation, below 2e-5
TOL_O = {torch.bfloat16: 3 * 2.0 ** -9, torch.float32: 2e-5}
TOL_S = 2e-5


def rel(x, ref) -> float:
    x, ref = x.detach().double().cpu(), ref.double()
    d = float(ref.norm())
    e = float((x - ref).norm())
    return e / d if d > 0 else e


def make(lens, H, Hk, dk, dv, dtype, seed=0, decay="token", h0=True, speed=1.0):
    """q, k, v, g, cu, h0; g between -speed and 0 with some tokens that keep everything."""
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    r = dict(generator=gen)
    q = torch.randn(T, Hk, dk, **r) * dk ** -0.5
    k = torch.randn(T, Hk, dk, **r) * dk ** -0.5
    v = torch.randn(T, H, dv, **r)
    if decay == "token":
        g = -speed * torch.rand(T, H, **r) * torch.rand(1, H, **r) ** 2
        g[torch.rand(T, H, **r) < 0.05] = 0.0
    else:
        g = -speed * torch.rand(H, **r) ** 3
    cu = torch.zeros(N + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(lens, dtype=torch.int64), 0).to(torch.int32)
    s = torch.randn(N, H, dk, dv, **r) * 0.3 if h0 else None
    return q.to(dtype), k.to(dtype), v.to(dtype), g, cu, s


def la_ref(q, k, v, g, cu, h0=None):
    """The recurrence, token by token."""
    T, H, dv = v.shape
    dk, N = q.shape[2], cu.numel() - 1
    rep = H // q.shape[1]
    q, k = (x.double().repeat_interleave(rep, 1) for x in (q, k))
    v, a = v.double(), g.double().exp().expand(T, H)
    S = torch.zeros(N, H, dk, dv, dtype=torch.float64) if h0 is None else h0.double().clone()
    o = torch.zeros(T, H, dv, dtype=torch.float64)
    for n in range(N):
        for t in range(int(cu[n]), int(cu[n + 1])):
            S[n] = S[n] * a[t][:, None, None] + k[t][:, :, None] * v[t][:, None, :]
            o[t] = torch.einsum("hij,hi->hj", S[n], q[t])
    return o, S


def qk_ref(x, positions, inv_freq, norm, layout, eps, weight, scale, rope_scale):
    x = x.double()
    D = x.shape[-1]
    if norm != "none":
        s = x.pow(2).sum(-1, keepdim=True)
        x = x / torch.sqrt((s / D if norm == "rms" else s) + eps)
    if weight is not None:
        x = x * weight.double()
    if inv_freq is not None:
        n = inv_freq.numel()
        ang = positions.double()[:, None] * inv_freq.double()[None, :]
        c, s = torch.cos(ang)[:, None] * rope_scale, torch.sin(ang)[:, None] * rope_scale
        y = x.clone()
        for i in range(n):
            a, b = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
            y[..., a] = x[..., a] * c[..., i] - x[..., b] * s[..., i]
            y[..., b] = x[..., b] * c[..., i] + x[..., a] * s[..., i]
        x = y
    return x * scale
