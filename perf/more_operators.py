"""Cases and plain forms of the paged half of a hybrid model's cache.

Layers with softmax attention keep the keys and values of every token, in pages that a block
table deals out to sequences, beside the fixed-size states of the linear layers:

  write   new keys and values into their pages, as they are or as e4m3 with one power-of-two
          scale a token and head
  read    tokens of the sequences gathered back from their pages
  chunk   attention of a chunk of new tokens a sequence over its whole paged context, causal,
          with an optional window and first tokens that stay visible
  decode  the same for one new token a sequence

Token i of the `len` new ones of sequence n stands at position kv_lens[n] - len + i, in slot
position % page_size of page block_table[n, position / page_size].

`run` computes a case in plain torch operations in 32 bits, rounded once at the end, or,
where `own` is true, through the library's entry points.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f32": 4, "e4m3": 1}
DEV = "cuda"


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # the keys and values of a 64-sequence decode step, pages of 16 tokens: latency
        dict(name="write_step", op="write", dtype="bf16", cache="e4m3", lens="step,64",
             before="uniform,64,100,4000", kv_heads=8, dim=128, page=16),
        # those of an 8192-token prompt
        dict(name="write_8k", op="write", dtype="bf16", cache="e4m3", lens="8192", before="0",
             kv_heads=8, dim=128, page=64),
        # a small model in single precision: three odd sequences, one of them empty
        dict(name="read_small_f32", op="read", dtype="f32", cache="f32", lens="37,0,513",
             before="5,70,0", kv_heads=3, dim=64, page=32),
        # the whole contexts of 16 sequences read back, as for moving them to another layout
        dict(name="read_packed", op="read", dtype="bf16", cache="e4m3",
             lens="uniform,16,512,4096", before="zeros,16", kv_heads=8, dim=128, page=64),
        # five short prompts and continuations (one of one token, one empty): latency
        dict(name="chunk_short", op="chunk", dtype="bf16", cache="bf16", lens="17,1,0,150,96",
             before="0,300,20,0,77", heads=8, kv_heads=2, dim=128, page=16, window=0, sinks=0),
        # one 8192-token prompt, 32 heads on 8
        dict(name="chunk_8k", op="chunk", dtype="bf16", cache="bf16", lens="8192", before="0",
             heads=32, kv_heads=8, dim=128, page=64, window=0, sinks=0),
        # 16 chunks that continue contexts of up to 4000 tokens, from a quantised cache
        dict(name="chunk_packed", op="chunk", dtype="bf16", cache="e4m3",
             lens="uniform,16,256,2048", before="uniform,16,0,4000", heads=32, kv_heads=8,
             dim=128, page=64, window=0, sinks=0),
        # the last 512 tokens of a long document: few rows, a long context
        dict(name="chunk_tail", op="chunk", dtype="bf16", cache="bf16", lens="512",
             before="65000", heads=32, kv_heads=8, dim=128, page=64, window=0, sinks=0),
        # a long prompt through a layer with a window of 1024 tokens and 4 sinks
        dict(name="chunk_window", op="chunk", dtype="bf16", cache="bf16", lens="16384",
             before="0", heads=16, kv_heads=4, dim=64, page=32, window=1024, sinks=4),
        # one sequence, one token: latency
        dict(name="decode_one", op="decode", dtype="bf16", cache="bf16", lens="step,1",
             before="2000", heads=32, kv_heads=8, dim=128, page=16, window=0, sinks=0),
        # a serving batch of 256 sequences, quantised cache
        dict(name="decode_256", op="decode", dtype="bf16", cache="e4m3", lens="step,256",
             before="uniform,256,512,8192", heads=32, kv_heads=8, dim=128, page=64, window=0,
             sinks=0),
        # four long documents
        dict(name="decode_long", op="decode", dtype="bf16", cache="bf16", lens="step,4",
             before="131072,131071,100000,90001", heads=32, kv_heads=8, dim=128, page=128,
             window=0, sinks=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "chunk", "chunk", "chunk", "chunk", "decode", "decode",
                     "decode"])
    dtype = rng.choice(["bf16"] * 5 + ["f32"])
    cache = rng.choice([dtype, dtype, "e4m3"])
    dim = rng.choice([128, 128, 64, 32])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 4, 5, 8, 16])
    case = dict(op=op, dtype=dtype, cache=cache, kv_heads=kv_heads, dim=dim,
                page=rng.choice([16, 32, 64, 128]))
    if op in ("write", "read"):
        count = _log(rng, 1, 64)
        total = _log(rng, 1, 16000)
        cuts = sorted(rng.randint(0, total) for _ in range(count - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        before = [rng.randint(0, 2000) for _ in lens]
    else:
        heads = kv_heads * group
        case.update(heads=heads, window=0, sinks=0)
        if rng.random() < 0.4:
            case.update(window=_log(rng, 1, 4000), sinks=rng.choice([0, 1, 4, 130]))
        if op == "decode":
            count = _log(rng, 1, 256)
            lens = None
            longest = _log(rng, 1, min(100000, 2000000 // count))
            before = [int(longest * rng.random()) for _ in range(count)]
        else:
            count = _log(rng, 1, 16)
            # at most the scores of the 8192-token prompt, 1/32 of it in single precision
            most = 8192 * 8192 * 32 // (32 if dtype == "f32" else 1)
            longest = _log(rng, 1, min(8192, math.isqrt(most // (heads * count))))
            lens = [rng.randint(0, longest) for _ in range(count)]
            lens[0] = longest
            context = max(longest, min(60000, most // (heads * longest * count)))
            before = [rng.randint(0, context - longest) for _ in lens]
    case["lens"] = "step,%d" % count if lens is None else ",".join(map(str, lens))
    case["before"] = ",".join(map(str, before))
    return case


def _numbers(text, rng=None):
    """"uniform,count,lo,hi" spreads whole numbers evenly over the range, in an order drawn
    from rng (they sum up to the same in every order)."""
    s = text.split(",")
    if s[0] == "step":
        return [1] * int(s[1])
    if s[0] == "zeros":
        return [0] * int(s[1])
    if s[0] != "uniform":
        return [int(x) for x in s]
    count, lo, hi = map(int, s[1:])
    v = [lo + (hi - lo) * (2 * i + 1) // (2 * count) for i in range(count)]
    return v if rng is None else [v[i] for i in rng.permutation(count)]


def _seen(a, b, window, sinks):
    """How many keys the tokens at positions a .. b - 1 see, each counted, and how many
    different ones."""
    pos = np.arange(a, b, dtype=np.int64)
    each = pos + 1
    if window:
        lo = np.maximum(0, pos - window + 1)
        each = pos + 1 - lo + np.minimum(lo, sinks)
        first = max(0, a - window + 1)
        distinct = b - first + min(first, sinks)
    else:
        distinct = b
    return int(each.sum()), int(distinct) if b > a else 0


def work(case):
    lens, before = _numbers(case["lens"]), _numbers(case["before"])
    Hk, D, T, N = case["kv_heads"], case["dim"], sum(lens), len(lens)
    b, c = SIZE[case["dtype"]], SIZE[case["cache"]]
    slot = 2 * Hk * (D * c + (4 if case["cache"] == "e4m3" else 0))   # keys and values of a token
    if case["op"] in ("write", "read"):
        return {"bytes": T * (2 * Hk * D * b + slot) + 12 * N + 4 * T // case["page"], "flops": 0}
    seen = [_seen(p, p + m, case["window"], case["sinks"]) for m, p in zip(lens, before)]
    H = case["heads"]
    return {"bytes": 2 * T * H * D * b + slot * sum(s[1] for s in seen) + 12 * N,
            "flops": 4 * D * H * sum(s[0] for s in seen)}


# --------------------------------------------------------------------------- inputs
def _scale_of(x):
    """The power of two that goes with a row: the least 2^e with max|x| / 2^e <= 448."""
    top = x.abs().amax(-1)
    part, e = torch.frexp(top)                   # top = part * 2^e, part in [0.5, 1)
    e = (e - 9 + (part > 0.875).int()).clamp(-100, 119)
    return torch.where(top > 0, torch.ldexp(torch.ones_like(top), e), torch.ones_like(top))


def _quantise(x):
    s = _scale_of(x)
    return (x / s[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rng = np.random.RandomState(seed % (1 << 31))
    f32 = dict(device=DEV, dtype=torch.float32, generator=gen)
    lens = _numbers(case["lens"], rng)
    before = _numbers(case["before"], rng)
    ctx = [a + b for a, b in zip(lens, before)]
    dt, ct, ps, Hk, D = DT[case["dtype"]], DT[case["cache"]], case["page"], case["kv_heads"], \
        case["dim"]
    s = {"op": case["op"], "longest": max(lens), "context": max(max(ctx), 1), "dtype": dt}

    def i32(x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)

    # pages dealt out in a random order, some left over; unused entries of the table are -1
    need = [-(-c // ps) for c in ctx]
    width = max(max(need), 1)
    pages = sum(need) + max(2, sum(need) // 16)
    order = rng.permutation(pages)
    table = np.full((len(ctx), width), -1, dtype=np.int64)
    at = 0
    for n, c in enumerate(need):
        table[n, :c] = order[at:at + c]
        at += c
    s["cu"] = i32(np.concatenate([[0], np.cumsum(lens)]))
    s["kv_lens"], s["table"] = i32(ctx), i32(table)
    s["total"] = sum(lens)
    # heads whose keys differ in size, as after a norm with weights
    size = 0.5 + torch.rand(Hk, 1, D, **f32)

    def fill(scale):
        x = torch.randn(pages, Hk, ps, D, **f32)
        if scale is not None:
            x *= scale
        if ct == torch.float8_e4m3fn:
            return _quantise(x)
        return x.to(ct), None

    s["k_pages"], s["k_scales"] = fill(size)
    s["v_pages"], s["v_scales"] = fill(None)
    T = sum(lens)
    if case["op"] == "write":
        # the output of one projection: keys and values side by side, some channels large
        x = torch.randn(T, 2 * Hk, D, **f32)
        x[:, :Hk] *= size[:, 0]
        x[..., :2] *= 8.0
        x = x.to(dt)
        s["k"], s["v"] = x[:, :Hk], x[:, Hk:]
    elif case["op"] != "read":
        H = case["heads"]
        # queries as they leave their preparation, scaled; some heads look around more sharply
        sharp = torch.exp2(2.0 * torch.rand(H, 1, **f32))
        s["q"] = (torch.randn(T, H, D, **f32) * (sharp * D ** -0.5)).to(dt)
        s["window"], s["sinks"] = case["window"], case["sinks"]
    return s


# ---------------------------------------------------------------------- plain forms
def _tokens(cu, kv_lens, total):
    """Sequence and position of each packed token."""
    t = torch.arange(total, device=cu.device)
    n = torch.searchsorted(cu[1:].contiguous(), t.to(cu.dtype), right=True)
    return n, kv_lens[n] - cu[n + 1] + t


def plain_write(s):
    n, pos = _tokens(s["cu"], s["kv_lens"], s["total"])
    ps = s["k_pages"].shape[2]
    page, slot = s["table"][n, pos // ps].long(), (pos % ps).long()
    for what in ("k", "v"):
        x, pages, scales = s[what].float(), s[what + "_pages"], s[what + "_scales"]
        if scales is None:
            pages[page, :, slot] = x.to(pages.dtype)
        else:
            x, scale = _quantise(x)
            pages.view(torch.uint8)[page, :, slot] = x.view(torch.uint8)
            scales[page, :, slot] = scale


def _values(pages, scales, at):
    """Pages (or slots of them) as the values they stand for."""
    if scales is None:
        return pages[at].float()
    return pages.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * scales[at][..., None]


def plain_read(s):
    n, pos = _tokens(s["cu"], s["kv_lens"], s["total"])
    ps = s["k_pages"].shape[2]
    at = (s["table"][n, pos // ps].long(), slice(None), (pos % ps).long())
    return tuple(_values(s[w + "_pages"], s[w + "_scales"], at).to(s["dtype"]) for w in "kv")


def plain_attention(s):
    """All sequences padded to the longest: scores of every new token against every key."""
    q, cu, kv_lens, L, M = s["q"], s["cu"].long(), s["kv_lens"].long(), s["context"], s["longest"]
    (T, H, D), N, Hk, ps = q.shape, cu.numel() - 1, s["k_pages"].shape[1], s["k_pages"].shape[2]
    key = torch.arange(L, device=q.device)
    there = key[None, :] < kv_lens[:, None]                               # [N, L]
    table = s["table"][:, :-(-L // ps)].clamp_min(0).long()

    def context(pages, scales):                                           # -> [N, Hk, L, D]
        x = _values(pages, scales, table).transpose(1, 2).flatten(2, 3)[:, :, :L]
        return x.masked_fill(~there[:, None, :, None], 0.0)

    i = torch.arange(M, device=q.device)
    new = cu[1:] - cu[:-1]
    row = torch.where(i[None, :] < new[:, None], cu[:-1, None] + i[None, :], T)   # [N, M]
    x = torch.cat([q.float(), torch.zeros(1, H, D, device=q.device)])[row]
    x = x.reshape(N, M, Hk, H // Hk, D).permute(0, 2, 3, 1, 4).flatten(2, 3)      # [N, Hk, G M, D]
    pos = ((kv_lens - new)[:, None] + i[None, :])[:, :, None]                     # [N, M, 1]
    seen = key <= pos
    if s["window"]:
        seen &= (key > pos - s["window"]) | (key < s["sinks"])
    score = (x @ context(s["k_pages"], s["k_scales"]).transpose(2, 3)).unflatten(2, (-1, M))
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = p.sum(-1, keepdim=True)
    o = p.flatten(2, 3) @ context(s["v_pages"], s["v_scales"])
    o = o.unflatten(2, (-1, M)) / torch.where(total > 0, total, torch.ones_like(total))
    out = torch.zeros(T + 1, H, D, device=q.device)
    out[row.reshape(-1)] = o.permute(0, 3, 1, 2, 4).reshape(N * M, H, D)
    return out[:T].to(q.dtype)


def run(s):
    op = s["op"]
    if own:
        from gated_delta_rule_43_gb300 import kda
        cache = (s["k_pages"], s["v_pages"], s["table"], s["kv_lens"])
        scales = dict(k_scales=s["k_scales"], v_scales=s["v_scales"])
        if op == "write":
            kda.kv_cache_write(s["k"], s["v"], *cache, s["cu"], **scales)
            return s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]
        if op == "read":
            return kda.kv_cache_read(*cache, s["cu"], total_tokens=s["total"], dtype=s["dtype"],
                                     **scales)
        if op == "chunk":
            return kda.paged_attn_fwd(s["q"], *cache, s["cu"], window=s["window"],
                                      sinks=s["sinks"], **scales)
        return kda.paged_attn_decode_step(s["q"], *cache, window=s["window"], sinks=s["sinks"],
                                          **scales)
    if op == "write":
        plain_write(s)
        return s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]
    return plain_read(s) if op == "read" else plain_attention(s)


# ------------------------------------------------------------------- 64-bit answers
def exact(case, seed):
    """From the definitions in 64 bits: slots one sequence after the other, attention one head
    after the other, a few hundred tokens at a time."""
    s = prepare(case, seed)
    op, ps, Hk, D = case["op"], case["page"], case["kv_heads"], case["dim"]
    cu, ctx, table = s["cu"].tolist(), s["kv_lens"].tolist(), s["table"].long()

    def stored(what):
        x = s[what + "_pages"].to(torch.float64)
        return x if s[what + "_scales"] is None else x * s[what + "_scales"].double()[..., None]

    if op == "write":
        out = []
        for what in ("k", "v"):
            pages, new = s[what + "_pages"].to(torch.float64), s[what].double()
            scales = s[what + "_scales"]
            if scales is not None:
                scales = scales.double()
                # the power of two at or above max|x| / 448, put together from its bits
                part, e = torch.frexp(new.abs().amax(-1) / 448.0)
                one = ((e - (part == 0.5).int() + 1023).long() << 52).view(torch.float64)
                new = new / one[..., None]
            for n, (a, b) in enumerate(zip(cu, cu[1:])):
                pos = torch.arange(ctx[n] - (b - a), ctx[n], device=DEV)
                page, slot = table[n][pos // ps], pos % ps
                pages[page, :, slot] = new[a:b]
                if scales is not None:
                    scales[page, :, slot] = one[a:b]
            out.append((pages, scales))
        return out[0][0], out[1][0], out[0][1], out[1][1]
    if op == "read":
        out = []
        for what in ("k", "v"):
            pages, rows = stored(what), []
            for n, (a, b) in enumerate(zip(cu, cu[1:])):
                pos = torch.arange(ctx[n] - (b - a), ctx[n], device=DEV)
                rows.append(pages[table[n][pos // ps], :, pos % ps])
            out.append(torch.cat(rows))
        return tuple(out)
    if work(case)["flops"] > 2e12:
        return None
    k, v, q = stored("k"), stored("v"), s["q"].double()
    o = torch.zeros_like(q)
    group = case["heads"] // Hk
    for n, (a, b) in enumerate(zip(cu, cu[1:])):
        if a == b:
            continue
        L, first = ctx[n], ctx[n] - (b - a)
        here = table[n][:-(-L // ps)]
        for h in range(Hk):
            keys, vals = k[here, h].reshape(-1, D)[:L], v[here, h].reshape(-1, D)[:L]
            for t in range(a, b, 512):
                e = min(b, t + 512)
                pos = first + torch.arange(t - a, e - a, device=DEV)
                lo = 0
                if case["window"]:
                    lo = max(0, first + t - a - case["window"] + 1)
                hi = first + e - a
                j = torch.cat([torch.arange(min(case["sinks"], lo), device=DEV),
                               torch.arange(lo, hi, device=DEV)])
                see = j[None, :] <= pos[:, None]
                if case["window"]:
                    see &= (pos[:, None] - j[None, :] < case["window"]) | (j < case["sinks"])
                w = torch.einsum("tgd,jd->gtj", q[t:e, h * group:(h + 1) * group], keys[j])
                w = torch.where(see, w, torch.full((), -math.inf, dtype=w.dtype, device=DEV))
                w = torch.softmax(w, -1)
                o[t:e, h * group:(h + 1) * group] = torch.einsum("gtj,jd->tgd", w, vals[j])
    return o
