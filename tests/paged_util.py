"""64-bit restatements of the paged cache and its attention from their formulas, one token after
the other, and random batches for them."""
from __future__ import annotations

import math

import torch

BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def quantise(x):
    """Rows of x as (e4m3, power-of-two scale)."""
    x = x.double()
    fine = x.abs().where(x.isfinite(), torch.zeros_like(x)).amax(-1)
    e = [math.frexp(t / 448.0) for t in fine.flatten().tolist()]
    e = [0 if m == 0 else min(119, max(-100, k - (m == 0.5))) for m, k in e]
    s = torch.tensor([2.0 ** k for k in e], dtype=torch.float64).reshape(fine.shape).to(x.device)
    y = (x / s[..., None]).clamp(-448, 448)      # (a NaN stays one)
    return y.float().to(E4M3), s.float()


def values(pages, scales):
    """A pool as the values it stands for."""
    return pages.double() if scales is None else pages.double() * scales.double()[..., None]


class Batch:
    """Sequences of lens[n] new tokens behind before[n] others, their pages dealt out at random;
    what no sequence uses is NaN, and so are table entries' pages past a sequence's end."""

    def __init__(self, lens, before, Hk, D, dtype, cache, ps=16, seed=0, device="cpu", halves=False,
                 spare=3):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.before = lens, before
        self.Hk, self.D, self.dtype, self.ps = Hk, D, dtype, ps
        ctx = [max(0, a + b) for a, b in zip(lens, before)]
        need = [-(-c // ps) for c in ctx]
        self.P = P = sum(need) + spare
        order = torch.randperm(P, generator=gen)
        N = len(lens)
        table = torch.full((N, max(need + [1]) + 1), 1 << 30, dtype=torch.int64)
        at = 0
        for n, c in enumerate(need):
            table[n, :c] = order[at:at + c]
            at += c
        self.rows = [torch.randn(c, 2 * Hk, D, generator=gen) for c in ctx]   # keys, values
        pool = torch.full((P, 2, Hk, ps, D), math.nan)
        for n, c in enumerate(ctx):
            for j in range(c):
                pool[table[n, j // ps], :, :, j % ps] = self.rows[n][j].reshape(2, Hk, D)
        scales = None
        if cache is E4M3:
            pool, scales = quantise(pool)
            scales[pool.float().isnan().any(-1)] = math.nan
        else:
            pool = pool.to(cache)
        dev = lambda t: None if t is None else t.to(device)  # noqa: E731
        pool, scales = dev(pool), dev(scales)
        if halves:    # views of one pool
            self.k_pages, self.v_pages = pool[:, 0], pool[:, 1]
            self.k_scales, self.v_scales = (None, None) if scales is None else (scales[:, 0], scales[:, 1])
        else:
            self.k_pages, self.v_pages = pool[:, 0].contiguous(), pool[:, 1].contiguous()
            self.k_scales, self.v_scales = (None, None) if scales is None else \
                (scales[:, 0].contiguous(), scales[:, 1].contiguous())
        self.table = dev(table.to(torch.int32))
        self.kv_lens = dev(torch.tensor(ctx, dtype=torch.int32))
        cu = [0]
        for m in lens:
            cu.append(cu[-1] + m)
        self.cu = dev(torch.tensor(cu, dtype=torch.int32))
        self.T = cu[-1]

    @property
    def cache(self):
        return self.k_pages, self.v_pages, self.table, self.kv_lens

    @property
    def scales(self):
        return dict(k_scales=self.k_scales, v_scales=self.v_scales)

    def queries(self, H, seed=1, sharp=2.0):
        gen = torch.Generator().manual_seed(seed)
        q = torch.randn(self.T, H, self.D, generator=gen) * (sharp * self.D ** -0.5)
        return q.to(self.dtype).to(self.table.device)


def places(b):
    """(row, sequence, position) of every token of the call."""
    cu, ctx = b.cu.tolist(), b.kv_lens.tolist()
    for n in range(len(ctx)):
        for i in range(cu[n + 1] - cu[n]):
            yield cu[n] + i, n, ctx[n] - (cu[n + 1] - cu[n]) + i


def attention(b, q, scale=1.0, window=0, sinks=0):
    """(o, size): the definition, and sum w |v| / sum w, which roundings of the weights scale with."""
    k, v = values(b.k_pages, b.k_scales), values(b.v_pages, b.v_scales)
    q = q.double()
    T, H, D = q.shape
    g = H // b.Hk
    o, size = torch.zeros_like(q), torch.zeros_like(q)
    ctx = b.kv_lens.tolist()
    cu = b.cu.tolist()
    for n, c in enumerate(ctx):
        m = cu[n + 1] - cu[n]
        if not m or not c:
            continue
        pages = b.table[n, :-(-c // b.ps)].long()
        keys = k[pages].transpose(0, 1).reshape(b.Hk, -1, D)[:, :c].repeat_interleave(g, 0)
        vals = v[pages].transpose(0, 1).reshape(b.Hk, -1, D)[:, :c].repeat_interleave(g, 0)
        pos = torch.arange(c - m, c, device=q.device)[:, None]
        j = torch.arange(c, device=q.device)[None, :]
        see = j <= pos
        if window:
            see = see & ((j > pos - window) | (j < sinks))
        # (keys and values that nobody sees may be anything)
        used = see.any(0)
        keys, vals = keys.clone(), vals.clone()
        keys[:, ~used], vals[:, ~used] = 0, 0
        s = torch.einsum("thd,hjd->htj", q[cu[n]:cu[n + 1]], keys) * scale
        s = s.masked_fill(~see, -math.inf)
        w = torch.nan_to_num(torch.softmax(s, -1), nan=0.0)
        o[cu[n]:cu[n + 1]] = torch.einsum("htj,hjd->thd", w, vals)
        size[cu[n]:cu[n + 1]] = torch.einsum("htj,hjd->thd", w, vals.abs())
    return o, size


def check_attention(got, b, q, scale=1.0, window=0, sinks=0):
    """Every value within what its roundings can make.  bf16: the output is rounded (2^-8 of it at
    most), and each weight is (2^-8 of it at most, so 2^-8 of sum w |v| / sum w, in the sum
    and once more through the weights' own sum when that is taken before the rounding).  fp32 adds up
    D products of a score and its exponential: an exponent of size up to 32 carries 2^-24 of
    itself a few times over, so weights are off by 32 * 2^-24 * 4 < 1e-5, in bf16 storage too."""
    want, size = attention(b, q, scale, window, sinks)
    got = got.double()
    assert got.isfinite().all()
    slack = 2.0 ** -8 * (want.abs() + size) if b.dtype is BF else 0.0
    off = (got - want).abs() - (slack + 2e-5 * size + 1e-30)
    assert off.max() <= 0, f"{off.max():.3e} over, at {torch.nonzero(off > 0)[:4].tolist()} of {tuple(off.shape)}"
