"""Cases and plain forms of the decayed linear-attention serving path.

Four operators belong together in a hybrid model's serving loop, around the same fixed-size
fp32 states [slots, H, dk, dv] that the delta-rule layer keeps:

  qk_prep   per-head norm of queries and keys, and their position rotation, in one pass
  prefill   linear attention with one decay per head, chunked over packed sequences:
              S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t
  decode    the same recurrence for one token a sequence, the state updated in place
  pool      forking slots of a state pool, and compacting it after sequences have ended

`run` computes a case in plain torch operations in 32 bits, rounded once at the end, or,
where `own` is true, through the library's entry points.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
DEV = "cuda"


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # five short prompts (one of one token, one empty) that arrive in one batch: latency
        dict(name="prefill_short", op="prefill", dtype="bf16", lens="17,1,0,150,96", heads=8,
             qk_heads=8, dk=128, dv=128, decay="token", h0=False),
        # one 8192-token prompt through 32 heads
        dict(name="prefill_8k", op="prefill", dtype="bf16", lens="8192", heads=32, qk_heads=32,
             dk=128, dv=128, decay="token", h0=False),
        # 16 packed prompts of 512 to 4096 tokens that continue from states, a fixed decay per
        # head and query/key heads shared by four value heads
        dict(name="prefill_packed", op="prefill", dtype="bf16", lens="uniform,16,512,4096",
             heads=32, qk_heads=8, dk=128, dv=128, decay="head", h0=True),
        # one long document, few heads
        dict(name="prefill_long", op="prefill", dtype="bf16", lens="65536", heads=16,
             qk_heads=16, dk=128, dv=128, decay="token", h0=False),
        # a small model in single precision, ragged, key size unlike value size
        dict(name="prefill_f32", op="prefill", dtype="f32", lens="1000,37,513", heads=4,
             qk_heads=4, dk=64, dv=128, decay="token", h0=True),
        # one sequence, one token: latency
        dict(name="decode_one", op="decode", dtype="bf16", n=1, slots=0, heads=32, qk_heads=32,
             dk=128, dv=128, decay="token"),
        # a serving batch of 256 sequences whose states lie in a pool of 300 slots
        dict(name="decode_256", op="decode", dtype="bf16", n=256, slots=300, heads=32,
             qk_heads=32, dk=128, dv=128, decay="token"),
        # an odd batch in single precision, shared query/key heads, fixed decay
        dict(name="decode_37_f32", op="decode", dtype="f32", n=37, slots=0, heads=16,
             qk_heads=4, dk=64, dv=128, decay="head"),
        # queries and keys of a 64-sequence decode step at scattered long positions, half of
        # each head rotated in neighbouring pairs, frequencies stretched for long contexts
        dict(name="qk_step", op="qk_prep", dtype="bf16", tokens=64, q_heads=32, k_heads=8,
             dim=128, rot=64, layout="interleaved", norm="rms", stretch=32.0, fused=True),
        # queries and keys of an 8192-token prompt, read from the fused projection's output
        dict(name="qk_8k", op="qk_prep", dtype="bf16", tokens=8192, q_heads=32, k_heads=32,
             dim=128, rot=128, layout="half", norm="l2", stretch=1.0, fused=True),
        # 12 prompts forked into 6 continuations each
        dict(name="pool_fork", op="pool_fork", slots=120, sources=12, copies=6, heads=32, dk=128,
             dv=128),
        # a pool whose sequences have ended here and there is packed to the front
        dict(name="pool_compact", op="pool_compact", slots=256, live=160, moved=60, heads=32,
             dk=128, dv=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "decode", "decode", "qk_prep", "qk_prep",
                     "pool_fork", "pool_compact"])
    qk = rng.choice([1, 2, 4, 8])
    heads = qk * rng.choice([1, 1, 2, 4])
    dk, dv = rng.choice([(128, 128), (128, 128), (128, 128), (64, 64), (64, 128), (128, 64),
                         (32, 32)])
    if op == "prefill":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        count = _log(rng, 1, 24)
        # at most the long case's 65536 x 16 token-heads; 1/64 of it in single precision
        most = 65536 * 16 // heads // (64 if dtype == "f32" else 1)
        total = _log(rng, 40, min(most, 60000))
        cuts = sorted(rng.randint(0, total) for _ in range(count - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        return dict(op=op, dtype=dtype, lens=",".join(map(str, lens)), heads=heads, qk_heads=qk,
                    dk=dk, dv=dv, decay=rng.choice(["token", "token", "head"]),
                    h0=rng.random() < 0.5)
    if op == "decode":
        n = _log(rng, 1, 256)
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), n=n,
                    slots=rng.choice([0, n + rng.randint(1, 40)]), heads=heads, qk_heads=qk,
                    dk=dk, dv=dv, decay=rng.choice(["token", "head"]))
    if op == "qk_prep":
        dim = rng.choice([128, 128, 64, 32])
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), tokens=_log(rng, 1, 16000),
                    q_heads=heads, k_heads=qk, dim=dim,
                    rot=rng.choice([r for r in (0, 16, 32, 48, 64, 96, 128) if r <= dim]),
                    layout=rng.choice(["half", "interleaved"]),
                    norm=rng.choice(["l2", "rms", "none"]), stretch=rng.choice([1.0, 4.0, 32.0]),
                    fused=rng.random() < 0.5)
    if op == "pool_fork":
        sources, copies = _log(rng, 1, 12), _log(rng, 1, 12)
        return dict(op=op, slots=sources * (copies + 1) + rng.randint(0, 40), sources=sources,
                    copies=copies, heads=heads, dk=dk, dv=dv)
    slots = _log(rng, 6, 280)
    live = max(1, int(slots * rng.uniform(0.2, 0.9)))
    return dict(op=op, slots=slots, live=live, moved=rng.randint(0, min(live, slots - live)),
                heads=heads, dk=dk, dv=dv)


def _lens(case, rng=None):
    """Lengths of the case's sequences.  "uniform,count,lo,hi" spreads them evenly over the
    range, in an order drawn from rng (they sum up to the same in every order)."""
    s = case["lens"].split(",")
    if s[0] != "uniform":
        return [int(x) for x in s]
    count, lo, hi = map(int, s[1:])
    lens = [lo + (hi - lo) * (2 * i + 1) // (2 * count) for i in range(count)]
    return lens if rng is None else [lens[i] for i in rng.permutation(count)]


def work(case):
    op = case["op"]
    if op == "prefill":
        lens = _lens(case)
        T, N = sum(lens), len(lens)
        H, Hk, dk, dv, b = case["heads"], case["qk_heads"], case["dk"], case["dv"], \
            SIZE[case["dtype"]]
        state = N * H * dk * dv * 4
        nbytes = T * (2 * Hk * dk + 2 * H * dv) * b + (T * H * 4 if case["decay"] == "token"
                                                       else H * 4)
        # the recurrence itself: an outer product and a matrix-vector product a token and head
        return {"bytes": nbytes + state * (2 if case["h0"] else 1), "flops": 4 * T * H * dk * dv}
    if op == "decode":
        n, H, Hk, dk, dv, b = case["n"], case["heads"], case["qk_heads"], case["dk"], \
            case["dv"], SIZE[case["dtype"]]
        return {"bytes": 2 * n * H * dk * dv * 4 + n * (2 * Hk * dk + 2 * H * dv) * b + n * H * 4,
                "flops": 5 * n * H * dk * dv}
    if op == "qk_prep":
        vals = case["tokens"] * (case["q_heads"] + case["k_heads"]) * case["dim"]
        return {"bytes": 2 * vals * SIZE[case["dtype"]] + case["tokens"] * 4, "flops": 7 * vals}
    slot = case["heads"] * case["dk"] * case["dv"] * 4
    if op == "pool_fork":
        return {"bytes": slot * case["sources"] * (1 + case["copies"]), "flops": 0}
    return {"bytes": 2 * slot * case["moved"] + case["slots"] * 5, "flops": 0}


# --------------------------------------------------------------------------- inputs
def _inv_freq(rot, stretch):
    """Rotation rates base^(-2i/rot) of a context that was stretched: rates whose period is
    long against the first context are divided by `stretch`, fast ones are kept, with a
    linear blend between them."""
    i = np.arange(rot // 2, dtype=np.float64)
    rate = 500000.0 ** (-2.0 * i / max(rot, 1))
    turns = 8192.0 * rate / (2.0 * math.pi)
    keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
    return (rate * (keep + (1.0 - keep) / stretch)).astype(np.float32)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rng = np.random.RandomState(seed % (1 << 31))
    f32 = dict(device=DEV, dtype=torch.float32, generator=gen)
    op = case["op"]
    s = {"op": op}

    def unit(x, scale=1.0):
        return x * (scale / x.norm(dim=-1, keepdim=True).clamp_min(1e-30))

    def slots_of(n, H, dk, dv):
        return torch.randn(n, H, dk, dv, **f32)

    if op in ("prefill", "decode"):
        dt = DT[case["dtype"]]
        H, Hk, dk, dv = case["heads"], case["qk_heads"], case["dk"], case["dv"]
        if op == "prefill":
            lens = _lens(case, rng)
            n = sum(lens)
            s["longest"] = max(lens)
            s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32,
                                   device=DEV)
        else:
            n = case["n"]
        s["q"] = unit(torch.randn(n, Hk, dk, **f32), dk ** -0.5).to(dt)
        s["k"] = unit(torch.randn(n, Hk, dk, **f32)).to(dt)
        s["v"] = torch.randn(n, H, dv, **f32).to(dt)
        # decays that keep a token for 1 to about 500 steps
        if case["decay"] == "head":
            s["g"] = -torch.exp2(-8.0 * torch.arange(1, H + 1, device=DEV) / H
                                 - torch.rand(H, **f32))
        else:
            s["g"] = -torch.exp(-6.0 * torch.rand(1, H, **f32)) * torch.rand(n, H, **f32)
        if op == "prefill":
            s["h0"] = 0.1 * slots_of(len(lens), H, dk, dv) if case["h0"] else None
        elif case["slots"]:
            s["state"] = 0.1 * slots_of(case["slots"], H, dk, dv)
            s["idx"] = torch.tensor(rng.permutation(case["slots"])[:n], dtype=torch.int32,
                                    device=DEV)
        else:
            s["state"], s["idx"] = 0.1 * slots_of(n, H, dk, dv), None
    elif op == "qk_prep":
        dt = DT[case["dtype"]]
        T, Hq, Hk, D = case["tokens"], case["q_heads"], case["k_heads"], case["dim"]
        if case["fused"]:  # the output of one projection: queries, keys and values side by side
            x = torch.randn(T, Hq + 2 * Hk, D, **f32).to(dt)
            s["q"], s["k"] = x[:, :Hq], x[:, Hq:Hq + Hk]
        else:
            s["q"] = torch.randn(T, Hq, D, **f32).to(dt)
            s["k"] = torch.randn(T, Hk, D, **f32).to(dt)
        if T <= 256:  # single tokens of sequences that are far apart
            pos = rng.randint(0, 1 << 20, T)
        else:
            pos = np.arange(T) + rng.randint(0, 1 << 19)
        s["pos"] = torch.tensor(pos, dtype=torch.int32, device=DEV)
        s["inv_freq"] = torch.tensor(_inv_freq(case["rot"], case["stretch"]), device=DEV)
        # the factor that goes with stretched rates
        s["rope_scale"] = 1.0 + 0.1 * math.log(case["stretch"])
        s["q_weight"] = s["k_weight"] = None
        if case["norm"] == "rms":
            s["q_weight"] = 1.0 + 0.1 * torch.randn(D, **f32)
            s["k_weight"] = 1.0 + 0.1 * torch.randn(D, **f32)
        s["norm"], s["layout"], s["q_scale"], s["eps"] = case["norm"], case["layout"], \
            D ** -0.5, 1e-6
    else:
        s["pool"] = slots_of(case["slots"], case["heads"], case["dk"], case["dv"])
        order = rng.permutation(case["slots"])
        if op == "pool_fork":
            n, c = case["sources"], case["copies"]
            s["src"] = torch.tensor(np.repeat(order[:n], c), dtype=torch.int32, device=DEV)
            s["dst"] = torch.tensor(order[n:n * (1 + c)], dtype=torch.int32, device=DEV)
        else:
            live = np.arange(case["slots"]) < case["live"]
            live[rng.permutation(case["live"])[:case["moved"]]] = False
            live[case["live"] + rng.permutation(case["slots"] - case["live"])[:case["moved"]]] \
                = True
            s["live"] = torch.tensor(live, device=DEV)
    return s


# ---------------------------------------------------------------------- plain forms
def _between(x):
    """[..., L] -> [..., L, L]: entry (t, s) is x_{s+1} + ... + x_t for t >= s, else -inf."""
    L = x.shape[-1]
    i = torch.arange(L, device=x.device)
    y = torch.where(i[:, None] > i[None, :], x[..., :, None], torch.zeros((), device=x.device))
    return y.cumsum(-2).masked_fill(i[:, None] < i[None, :], -math.inf)


def plain_prefill(q, k, v, g, cu, h0, longest):
    """The chunked form: dense products inside 64-token chunks, the chunks' start states as
    one product of all chunks' contributions with the decays between them."""
    C, (T, H, dv), dk, N = 64, v.shape, q.shape[-1], cu.numel() - 1
    nc = -(-longest // C)
    at = torch.arange(nc * C, device=q.device)
    begin, length = cu[:-1].long(), (cu[1:] - cu[:-1]).long()
    here = at[None, :] < length[:, None]                             # [N, nc*C]
    row = torch.where(here, begin[:, None] + at[None, :], T)         # T: a row of zeros

    def padded(x):                                                   # -> [N, nc, H, C, D]
        x = torch.cat([x.float(), x.new_zeros(1, *x.shape[1:], dtype=torch.float32)])[row]
        x = x.reshape(N, nc, C, *x.shape[2:]).transpose(2, 3)
        return x.repeat_interleave(H // x.shape[2], dim=2)
    q, k, v = padded(q), padded(k), padded(v)
    g = padded(g.float().expand(T, H)[..., None])[..., 0]            # [N, nc, H, C]
    p = (q @ k.transpose(-1, -2)) * _between(g).exp()
    o = p @ v
    after = (g.flip(-1).cumsum(-1).flip(-1) - g).exp()               # decay to the chunk's end
    add = (k * after[..., None]).transpose(-1, -2) @ v               # [N, nc, H, dk, dv]
    # start states: chunk c's is the sum over earlier ones, entry 0 the initial state
    s0 = torch.zeros(N, 1, H, dk, dv, device=q.device) if h0 is None else h0[:, None]
    every = torch.cat([s0, add], 1).permute(0, 2, 1, 3, 4).reshape(N, H, nc + 1, dk * dv)
    total = torch.cat([torch.zeros_like(g[:, :1, :, 0]), g.sum(-1)], 1).transpose(1, 2)
    start = (_between(total).exp() @ every).reshape(N, H, nc + 1, dk, dv).transpose(1, 2)
    o = o + (q * g.cumsum(-1).exp()[..., None]) @ start[:, :-1]
    out = o.new_zeros(T + 1, H, dv)
    out[row.reshape(-1)] = o.transpose(2, 3).reshape(N * nc * C, H, dv)
    return out[:T], start[:, -1].contiguous()


def plain_decode(q, k, v, g, state, idx):
    H = v.shape[1]
    q, k = (x.float().repeat_interleave(H // x.shape[1], dim=1) for x in (q, k))
    S = state if idx is None else state[idx.long()]
    S = S * g.exp().expand(v.shape[:2])[..., None, None] + k[..., None] * v.float()[:, :, None]
    if idx is None:
        state.copy_(S)
    else:
        state[idx.long()] = S
    return (S * q[..., None]).sum(2)


def plain_qk(x, weight, pos, inv_freq, norm, eps, scale, layout, rope_scale):
    x = x.float()
    if norm != "none":
        x2 = x.square()
        x = x * ((x2.sum(-1, keepdim=True) if norm == "l2" else x2.mean(-1, keepdim=True))
                 + eps).rsqrt()
    if weight is not None:
        x = x * weight
    rot = 2 * inv_freq.numel()
    # angles over many turns: reduced in 64 bits, the rest in 32
    turn = pos.double()[:, None] * inv_freq.double() / (2.0 * math.pi)
    angle = ((turn - turn.floor()) * (2.0 * math.pi)).float()[:, None, :]
    cos, sin = angle.cos() * rope_scale, angle.sin() * rope_scale
    head, rest = x[..., :rot], x[..., rot:]
    if layout == "half":
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        head = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([head, rest], -1) * scale


def plain_compact(pool, live):
    at = torch.arange(live.numel(), device=live.device)
    n = live.sum()
    src, dst = at[live & (at >= n)], at[~live & (at < n)]   # both ascending, one to one
    index = torch.where(live, at, -1)
    index[src] = dst
    pool[dst] = pool[src]
    return pool, index.to(torch.int32), n.to(torch.int32).reshape(1)


def run(s):
    op = s["op"]
    if own:
        from gated_delta_rule_43_gb300 import kda
        if op == "prefill":
            return kda.la_chunk_fwd(s["q"], s["k"], s["v"], s["g"], s["cu"], s["h0"])
        if op == "decode":
            if s["idx"] is None:
                return kda.la_decode_step(s["q"], s["k"], s["v"], s["g"], s["state"]), s["state"]
            return kda.la_decode_step_indexed(s["q"], s["k"], s["v"], s["g"], s["state"],
                                              s["idx"]), s["state"]
        if op == "qk_prep":
            return kda.qk_norm_rope(s["q"], s["k"], s["pos"], s["inv_freq"], norm=s["norm"],
                                    layout=s["layout"], eps=s["eps"], q_weight=s["q_weight"],
                                    k_weight=s["k_weight"], q_scale=s["q_scale"],
                                    rope_scale=s["rope_scale"])
        if op == "pool_fork":
            kda.state_pool_copy(s["pool"], s["src"], s["dst"])
            return s["pool"]
        return (s["pool"],) + tuple(kda.state_pool_compact(s["pool"], s["live"]))
    if op == "prefill":
        o, last = plain_prefill(s["q"], s["k"], s["v"], s["g"], s["cu"], s["h0"], s["longest"])
        return o.to(s["v"].dtype), last
    if op == "decode":
        o = plain_decode(s["q"], s["k"], s["v"], s["g"], s["state"], s["idx"])
        return o.to(s["v"].dtype), s["state"]
    if op == "qk_prep":
        common = (s["pos"], s["inv_freq"], s["norm"], s["eps"])
        tail = (s["layout"], s["rope_scale"])
        return (plain_qk(s["q"], s["q_weight"], *common, s["q_scale"], *tail).to(s["q"].dtype),
                plain_qk(s["k"], s["k_weight"], *common, 1.0, *tail).to(s["k"].dtype))
    if op == "pool_fork":
        s["pool"][s["dst"].long()] = s["pool"][s["src"].long()]
        return s["pool"]
    return plain_compact(s["pool"], s["live"])


# ------------------------------------------------------------------- 64-bit answers
def exact(case, seed):
    """From the definitions: the recurrence token by token, rotation as a complex product,
    slots moved one at a time; all in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op in ("prefill", "decode"):
        v, H = s["v"].double(), case["heads"]
        group = torch.arange(H, device=DEV) // (H // case["qk_heads"])
        q, k = s["q"].double()[:, group], s["k"].double()[:, group]
        a = s["g"].double().exp().expand(v.shape[:2])
        if op == "decode":
            at = torch.arange(case["n"], device=DEV) if s["idx"] is None else s["idx"].long()
            state = s["state"].double()
            S = torch.einsum("nh,nhij->nhij", a, state[at]) + torch.einsum("nhi,nhj->nhij", k, v)
            state[at] = S
            return torch.einsum("nhij,nhi->nhj", S, q), state
        cu = s["cu"].tolist()
        lens = [e - b for b, e in zip(cu, cu[1:])]
        if sum(lens) * H * case["dk"] * case["dv"] > 3e10:
            return None
        by_length = sorted(range(len(lens)), key=lambda n: -lens[n])
        begin = torch.tensor([cu[n] for n in by_length], device=DEV)
        S = torch.zeros(len(lens), H, case["dk"], case["dv"], dtype=torch.float64, device=DEV)
        if s["h0"] is not None:
            S = s["h0"].double()[by_length]
        o = torch.zeros_like(v)
        alive = len(lens)
        for t in range(max(lens)):
            while alive and lens[by_length[alive - 1]] <= t:
                alive -= 1
            i = begin[:alive] + t
            S[:alive] *= a[i][:, :, None, None]
            S[:alive] += k[i].unsqueeze(-1) * v[i].unsqueeze(-2)
            o[i] = torch.matmul(q[i].unsqueeze(-2), S[:alive]).squeeze(-2)
        last = torch.empty_like(S)
        last[by_length] = S
        return o, last
    if op == "qk_prep":
        rate = s["inv_freq"].double()
        turn = torch.polar(torch.full((), s["rope_scale"], dtype=torch.float64, device=DEV),
                           s["pos"].double()[:, None] * rate)[:, None]
        got = []
        for x, w, scale in ((s["q"], s["q_weight"], s["q_scale"]), (s["k"], s["k_weight"], 1.0)):
            x = x.double()
            size = {"none": None, "l2": 1, "rms": x.shape[-1]}[s["norm"]]
            if size:
                x = x / (x.pow(2).sum(-1, keepdim=True) / size + s["eps"]).sqrt()
            x = x * scale if w is None else x * w.double() * scale
            n = rate.numel()
            pair = x[..., :2 * n].reshape(*x.shape[:2], *((2, n) if s["layout"] == "half"
                                                          else (n, 2)))
            dim = -2 if s["layout"] == "half" else -1
            z = torch.complex(pair.select(dim, 0), pair.select(dim, 1)) * turn
            x[..., :2 * n] = torch.stack([z.real, z.imag], dim).reshape(*x.shape[:2], 2 * n)
            got.append(x)
        return tuple(got)
    pool = s["pool"].double()
    if op == "pool_fork":
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            pool[b] = pool[a]
        return pool
    live = s["live"].tolist()
    holes = [i for i in range(sum(live)) if not live[i]]
    movers = [i for i in range(sum(live), len(live)) if live[i]]
    for a, b in zip(movers, holes):
        pool[b] = pool[a]
    return pool, None, None
