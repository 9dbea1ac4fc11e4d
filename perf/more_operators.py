"""Positions and chunks around the paged cache, as they are called in a decoder block, and their plain forms in
elementary torch operations.

rotate   queries and keys turned by their positions (Rotary.apply)
norm     the same behind a norm of each head, in one pass (Rotary.apply with weights)
append   new keys normed, turned and written to their pages beside the values, the queries of the same tokens normed
         and turned (KVCache.append)
chunk    attention of a chunk of new tokens of each sequence over the paged cache (Attention.chunk)

Rotation: pair p of the first `rot` elements of a head, (x[p], x[p + rot / 2]) in the half layout and (x[2p], x[2p + 1])
in the interleaved one, turns by the angle position * f_p, f_p = base^(-2p / rot), changed for long contexts:
  linear   f / factor
  base     base * factor^(rot / (rot - 2)) for base
  turns    n = original * f / 2 pi turns over the trained length: f (s + (1 - s) / factor) with s = (n - 1) / 3, cut to
           [0, 1] (low 1, high 4)
  pairs    f (1 - r + r / factor) with r rising from 0 to 1 between the pairs that make 32 and 1 turns over the trained
           length, rounded outwards; cosine and sine times 0.1 ln factor + 1
Norm: x / sqrt(mean x^2 + eps) * weight over the head, before the rotation.
Pool: k, v [layers][pages][kv_heads][page][dim]; table [slots][width], lens [slots], refs [pages].
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_DEV = "cuda"
_EPS = 1e-6


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step's queries and keys of eight sequences far into their contexts, where launch latency counts
        dict(name="rotate_step", op="rotate", tokens=8, seqs=8, far=131072, heads=32, kv_heads=8, dim=128, rot=128,
             layout="half", scaling="none", factor=1.0, original=0, base=10000.0, dtype="bf16", pick=1),
        # a prefill of 16384 tokens at d = 4096 (32 heads of 128) whose context is eight times the trained one
        dict(name="rotate_prefill", op="rotate", tokens=16384, seqs=3, far=16384, heads=32, kv_heads=8, dim=128, rot=128,
             layout="half", scaling="pairs", factor=8.0, original=4096, base=10000.0, dtype="bf16", pick=2),
        # fp32 heads of odd size of which two fifths turn, neighbours as pairs
        dict(name="rotate_part", op="rotate", tokens=1001, seqs=5, far=4000, heads=6, kv_heads=3, dim=80, rot=32,
             layout="interleaved", scaling="linear", factor=4.0, original=0, base=10000.0, dtype="f32", pick=3),
        # a decode step of 64 sequences at d = 8192 (64 heads of 128)
        dict(name="norm_step", op="norm", tokens=64, seqs=64, far=32768, heads=64, kv_heads=8, dim=128, rot=128,
             layout="half", scaling="turns", factor=8.0, original=8192, base=500000.0, dtype="bf16", pick=4),
        # the largest prefill of a layer at d = 8192
        dict(name="norm_prefill", op="norm", tokens=16384, seqs=1, far=0, heads=64, kv_heads=8, dim=128, rot=128,
             layout="half", scaling="none", factor=1.0, original=0, base=1000000.0, dtype="bf16", pick=5),
        # ragged fp32 prompts of small heads
        dict(name="norm_ragged", op="norm", tokens=777, seqs=13, far=0, heads=16, kv_heads=4, dim=64, rot=64,
             layout="interleaved", scaling="base", factor=4.0, original=0, base=10000.0, dtype="f32", pick=6),
        # a decode step's new token of 64 sequences, d = 8192
        dict(name="append_step", op="append", seqs=64, base_len=8192, new=64, heads=64, kv_heads=8, dim=128, rot=128,
             layout="half", scaling="none", factor=1.0, original=0, base=10000.0, norm=True, page=64, dtype="bf16", pick=7),
        # eight prompts admitted together
        dict(name="append_prompt", op="append", seqs=8, base_len=0, new=16384, heads=32, kv_heads=8, dim=128, rot=128,
             layout="half", scaling="none", factor=1.0, original=0, base=10000.0, norm=True, page=64, dtype="bf16", pick=8),
        # drafted tokens of 31 fp32 sequences, neighbours as pairs, no norm
        dict(name="append_draft", op="append", seqs=31, base_len=2000, new=160, heads=8, kv_heads=2, dim=64, rot=64,
             layout="interleaved", scaling="linear", factor=2.0, original=0, base=10000.0, norm=False, page=16, dtype="f32",
             pick=9),
        # a tiny fp32 layer's 40 tokens of three sequences, where launch latency counts
        dict(name="chunk_small", op="chunk", seqs=3, new=40, kind="even", past=100, heads=4, kv_heads=2, dim=32, page=16,
             dtype="f32", pick=10),
        # a serving step of 64 sequences: most with one token or a few drafted ones, some with a piece of their prompt
        dict(name="chunk_mixed", op="chunk", seqs=64, new=2100, kind="mixed", past=16384, heads=64, kv_heads=8, dim=128,
             page=64, dtype="bf16", pick=11),
        # the last piece of a long prompt: 4096 tokens behind 28672
        dict(name="chunk_long", op="chunk", seqs=1, new=4096, kind="even", past=28672, heads=32, kv_heads=8, dim=128,
             page=64, dtype="bf16", pick=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "norm", "append", "append", "chunk", "chunk", "chunk"])
    kv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([g for g in (1, 2, 3, 4, 6, 8) if g * kv <= 64])
    dim = rng.choice([64, 64, 128, 128, 128, 32, 80, 96, 256])
    f32 = rng.random() < 0.25
    c = dict(op=op, heads=kv * group, kv_heads=kv, dim=dim, dtype="f32" if f32 else "bf16", pick=rng.randrange(1 << 20))
    if op != "chunk":
        rot = rng.choice([dim, dim, dim, dim // 2, dim // 4])
        scaling = rng.choice(["none", "none", "linear", "base", "turns", "pairs"])
        c.update(rot=rot, layout=rng.choice(["half", "half", "interleaved"]), scaling=scaling,
                 factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]),
                 original=rng.choice([2048, 4096, 8192]) if scaling in ("turns", "pairs") else 0,
                 base=rng.choice([10000.0, 10000.0, 500000.0, 1000000.0]))
    # tokens of at most as many elements as the largest listed case of the operator has
    width = (c["heads"] + (1 if op in ("rotate", "norm") else 2) * kv) * dim * (2 if f32 else 1)
    if op in ("rotate", "norm"):
        tokens = _log_int(rng, 1, min(16384, (16384 * (40 if op == "rotate" else 72) * 128) // width))
        c.update(tokens=tokens, seqs=min(tokens, _log_int(rng, 1, 64)), far=rng.choice([0, _log_int(rng, 1, 1 << 20)]))
        return c
    c["page"] = rng.choice([16, 32, 64, 128, 256])
    if op == "append":
        n = _log_int(rng, 1, 64)
        most = (16384 * 48 * 128) // width
        c.update(seqs=n, base_len=rng.choice([0, _log_int(rng, 1, 4096)]), new=min(most, n * _log_int(rng, 1, 256) + rng.randrange(n)),
                 norm=rng.random() < 0.5)
        return c
    kind = rng.choice(["even", "draft", "mixed"])
    if kind == "even":  # pieces of prompts
        n = _log_int(rng, 1, 8)
        new, past = _log_int(rng, n, 512 if f32 else 4096), rng.choice([0, _log_int(rng, 1, 2048 if f32 else 16384)])
    elif kind == "draft":  # one to eight tokens of each sequence
        n = _log_int(rng, 1, 64)
        new, past = n * rng.randint(1, 8), _log_int(rng, 1, 1024 if f32 else 16384)
    else:
        n = _log_int(rng, 2, 64)
        new, past = n * 4 + _log_int(rng, 1, 128 if f32 else 1024), _log_int(rng, 1, 1024 if f32 else 8192)
    # (a large head's or batch's sequences are shorter: at most the largest listed case's work)
    past = min(past, (1 << 41) // (4 * new * c["heads"] * dim), (1 << 32) // (4 * n * kv * dim))
    c.update(seqs=n, new=new, kind=kind, past=past)
    return c


def _parts(total, count, pick):
    """`count` lengths of very different size that sum to `total` (each at least 1 where total allows it)."""
    r = random.Random(pick)
    w = [r.expovariate(1.0) ** 1.5 + 1e-3 for _ in range(count)]
    base = 1 if total >= count else 0
    left = total - base * count
    n = [base + int(left * x / sum(w)) for x in w]
    n[r.randrange(count)] += total - sum(n)
    return n


def _starts(case):
    """Lengths and first positions of a rotate or norm case's sequences."""
    n = _parts(case["tokens"], case["seqs"], case["pick"])
    r = random.Random(case["pick"] + 1)
    return n, [r.randint(0, case["far"]) for _ in n]


def _grown(case):
    """Positions held before and new tokens of an append case's sequences."""
    r = random.Random(case["pick"])
    return [r.randint(0, case["base_len"]) for _ in range(case["seqs"])], _parts(case["new"], case["seqs"], case["pick"])


def _chunks(case):
    """New tokens and positions held altogether of a chunk case's sequences."""
    n, new, r = case["seqs"], case["new"], random.Random(case["pick"])
    if case["kind"] == "mixed":  # an eighth have a piece of a prompt, the others one to four tokens
        few = [r.choice([1, 1, 1, 2, 4]) for _ in range(n)]
        long = max(1, n // 8)
        nq = [a + b for a, b in zip(few, _parts(new - sum(few), long, case["pick"]) + [0] * (n - long))]
        r.shuffle(nq)
    elif case["kind"] == "draft":
        nq = [new // n + (i < new % n) for i in range(n)]
    else:
        nq = _parts(new, n, case["pick"])
    past = [case["past"]] + [r.randint(0, case["past"]) for _ in range(n - 1)]
    return nq, [a + b for a, b in zip(nq, past)]


def _up(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device=_DEV, dtype=torch.float32).to(dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=_DEV)


def _offsets(lens):
    o = [0]
    for a in lens:
        o.append(o[-1] + a)
    return o


def _frequencies(case):
    """(f_p in radians a position, the factor of cosine and sine), 64 bits."""
    R, base, factor = case["rot"], case["base"], case["factor"]
    if case["scaling"] == "base":
        base = base * factor ** (R / (R - 2))
    p = torch.arange(R // 2, dtype=torch.float64)
    f, magnitude = base ** (-2 * p / R), 1.0
    if case["scaling"] == "linear":
        f = f / factor
    elif case["scaling"] == "turns":
        s = ((case["original"] * f / (2 * math.pi) - 1) / 3).clamp(0, 1)
        f = f * (s + (1 - s) / factor)
    elif case["scaling"] == "pairs":
        def pair(turns):
            return R * math.log(case["original"] / (2 * math.pi * turns)) / (2 * math.log(base))
        lo, hi = max(0, math.floor(pair(32))), min(R - 1, math.ceil(pair(1)))
        r = ((p - lo) / (hi - lo if hi > lo else 0.001)).clamp(0, 1)
        f, magnitude = f * (1 - r + r / factor), 0.1 * math.log(factor) + 1
    return f.to(_DEV), magnitude


def _rotary(case):
    import sparse_mixture_experts_moe_gb300 as moe
    more = dict(low=1.0, high=4.0) if case["scaling"] == "turns" else dict(low=1.0, high=32.0) if case["scaling"] == "pairs" else {}
    return moe.Rotary(case["dim"], rotary_dim=case["rot"], base=case["base"], layout=case["layout"],
                      scaling=None if case["scaling"] == "none" else case["scaling"], factor=case["factor"],
                      original_len=case["original"], **more)


def _table(rows, width):
    return _ints([r + [-1] * (width - len(r)) for r in rows])


def _cache_state(case, g, rows, lens, pages, width):
    shape = (1, pages, case["kv_heads"], case["page"], case["dim"])
    t = _TYPES[case["dtype"]]
    k, v = (torch.randn(shape, generator=g, device=_DEV, dtype=t) for _ in range(2))
    v += 0.5 * torch.randn((case["dim"],), generator=g, device=_DEV).to(t)
    st = dict(k=k, v=v, table=_table(rows, width), lens=_ints(lens),
              refs=_ints([0] * pages).index_fill_(0, _ints([p for r in rows for p in r]).long(), 1), page=case["page"])
    if own:  # the handle that a user's program keeps for its cache
        import sparse_mixture_experts_moe_gb300 as moe
        st["cache"] = moe.KVCache(st["k"], st["v"], st["table"], st["lens"], st["refs"])
    return st


def _pages(lens, page, seed):
    """Pages of slots that hold `lens` positions, as churn leaves them, in a pool with five free ones."""
    need = [_up(a, page) for a in lens]
    order = list(range(sum(need) + 5))
    random.Random(seed).shuffle(order)
    rows, at = [], 0
    for a in need:
        rows.append(order[at:at + a])
        at += a
    return rows, len(order)


def prepare(case, seed):
    g = _gen(seed)
    op, H, Hk, D, t = case["op"], case["heads"], case["kv_heads"], case["dim"], _TYPES[case["dtype"]]
    if op == "chunk":
        nq, nk = _chunks(case)
        rows, pages = _pages(nk, case["page"], seed)
        st = _cache_state(case, g, rows, nk, pages, _up(max(nk), case["page"]) + 1)
        x = _normal(g, (sum(nq), H + 2 * Hk, D), t)
        st.update(op=op, q=x[:, :H], slots=_ints(list(range(len(nq)))), offsets=_ints(_offsets(nq)), nq=nq, nk=nk,
                  scale=D ** -0.5)
        if own:
            import sparse_mixture_experts_moe_gb300 as moe
            st["attention"] = moe.Attention(H, Hk, D, t)
        return st
    if op == "append":
        held, new = _grown(case)
        total = [a + b for a, b in zip(held, new)]
        rows, pages = _pages(total, case["page"], seed)
        st = _cache_state(case, g, rows, total, pages, _up(max(total), case["page"]) + 1)
        st.update(slots=_ints(list(range(len(new)))), offsets=_ints(_offsets(new)), base=_ints(held))
        tokens = sum(new)
    else:
        n, start = _starts(case)
        st = dict(positions=torch.cat([torch.arange(a, device=_DEV, dtype=torch.int32) + s for a, s in zip(n, start)]))
        tokens = sum(n)
    # q, k and v as slices of one fused projection of the tokens
    x = _normal(g, (tokens, H + 2 * Hk, D), t)
    st.update(op=op, q=x[:, :H], xk=x[:, H:H + Hk], xv=x[:, H + Hk:], rot=case["rot"], layout=case["layout"], wq=None, wk=None)
    if op == "norm" or case.get("norm"):
        st.update(wq=(1 + 0.2 * torch.randn((D,), generator=g, device=_DEV)).to(t),
                  wk=(1 + 0.2 * torch.randn((D,), generator=g, device=_DEV)).to(t))
    if own:
        st["rotary"] = _rotary(case)
    else:
        st["freq"], st["magnitude"] = _frequencies(case)
    return st


# ---------------------------------------------------------------------------------------------- one pass

def run(st):
    return _OWN[st["op"]](st) if own else _PLAIN[st["op"]](st)


def _own_rotate(st):
    return st["rotary"].apply(st["q"], st["positions"], st["xk"])


def _own_norm(st):
    return st["rotary"].apply(st["q"], st["positions"], st["xk"], q_weight=st["wq"], k_weight=st["wk"], eps=_EPS)


def _own_append(st):
    q = st["cache"].append(st["xk"], st["xv"], st["slots"], st["offsets"], st["base"], st["rotary"], q=st["q"],
                           q_weight=st["wq"], k_weight=st["wk"], eps=_EPS)
    return [q, st["k"], st["v"]]


def _own_chunk(st):
    return st["attention"].chunk(st["q"], st["cache"], st["slots"], st["offsets"])


_OWN = {"rotate": _own_rotate, "norm": _own_norm, "append": _own_append, "chunk": _own_chunk}


def _angles(st, positions):
    a = positions.double()[:, None] * st["freq"]
    return (torch.cos(a) * st["magnitude"]).float()[:, None], (torch.sin(a) * st["magnitude"]).float()[:, None]


def _turn(st, x, weight, cos, sin):
    """x [tokens, heads, dim] normed (where there is a weight) and turned, 32 bits."""
    y, R = x.float(), st["rot"]
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + _EPS) * weight.float()
    if st["layout"] == "half":
        a, b = y[..., :R // 2], y[..., R // 2:R]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., R:]], -1)
    a, b = y[..., :R:2], y[..., 1:R:2]
    z = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([z, y[..., R:]], -1)


def _plain_rotate(st):
    cos, sin = _angles(st, st["positions"])
    return _turn(st, st["q"], st["wq"], cos, sin).to(st["q"].dtype), _turn(st, st["xk"], st["wk"], cos, sin).to(st["q"].dtype)


def _plain_append(st):
    o = st["offsets"].long()
    t = torch.arange(st["xk"].shape[0], device=_DEV)
    i = (t[:, None] >= o[None, 1:]).sum(1)
    p = st["base"].long()[i] + t - o[i]
    cos, sin = _angles(st, p)
    at = st["table"][st["slots"].long()[i], p // st["page"]].long()
    st["k"][0].transpose(1, 2)[at, p % st["page"]] = _turn(st, st["xk"], st["wk"], cos, sin).to(st["k"].dtype)
    st["v"][0].transpose(1, 2)[at, p % st["page"]] = st["xv"]
    return [_turn(st, st["q"], st["wq"], cos, sin).to(st["q"].dtype), st["k"], st["v"]]


def _plain_chunk(st):
    q, out, page = st["q"], torch.empty(st["q"].shape, dtype=st["q"].dtype, device=_DEV), st["page"]
    H, D, Hk = q.shape[1], q.shape[2], st["k"].shape[2]
    G, t0 = H // Hk, 0
    for s, (nq, nk) in enumerate(zip(st["nq"], st["nk"])):
        at = st["table"][st["slots"][s], :_up(nk, page)].long()
        k, v = (st[x][0, at].transpose(0, 1).reshape(Hk, -1, D)[:, :nk].float() for x in "kv")
        x = q[t0:t0 + nq].float().view(nq, Hk, G, D).permute(1, 2, 0, 3).reshape(Hk, G * nq, D) * st["scale"]
        hidden = torch.arange(nk, device=_DEV) > torch.arange(nk - nq, nk, device=_DEV)[:, None]
        for h in range(0, Hk, max(1, (1 << 29) // (G * nq * nk))):
            e = min(Hk, h + max(1, (1 << 29) // (G * nq * nk)))
            w = (x[h:e] @ k[h:e].transpose(1, 2)).view(e - h, G, nq, nk)
            w.masked_fill_(hidden, float("-inf"))
            w -= w.amax(-1, keepdim=True)
            w.exp_()
            o = (w.view(e - h, G * nq, nk) @ v[h:e]).view(e - h, G, nq, D) / w.sum(-1, keepdim=True)
            out[t0:t0 + nq].view(nq, Hk, G, D)[:, h:e] = o.permute(2, 0, 1, 3).to(out.dtype)
        t0 += nq
    return out


_PLAIN = {"rotate": _plain_rotate, "norm": _plain_rotate, "append": _plain_append, "chunk": _plain_chunk}


# ---------------------------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, eb, D, H, Hk = case["op"], 4 if case["dtype"] == "f32" else 2, case["dim"], case["heads"], case["kv_heads"]
    if op == "chunk":
        nq, nk = _chunks(case)
        pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(nq, nk))
        return {"bytes": (2 * sum(nq) * H + 2 * sum(nk) * Hk) * D * eb + 4 * sum(_up(b, case["page"]) for b in nk),
                "flops": 4 * D * H * pairs}
    norm = 4 if op == "norm" or case.get("norm") else 0
    if op == "append":
        tokens = case["new"]
        return {"bytes": 2 * tokens * (H + 2 * Hk) * D * eb, "flops": tokens * (H + Hk) * (3 * case["rot"] + norm * D)}
    tokens = case["tokens"]
    return {"bytes": 2 * tokens * (H + Hk) * D * eb + 4 * tokens, "flops": tokens * (H + Hk) * (3 * case["rot"] + norm * D)}


# ---------------------------------------------------------------------------------------------- from the definitions, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "chunk":
        return _exact_chunk(st)
    if case["op"] != "append":
        p = st["positions"].double()
        return tuple(_exact_heads(case, st[x], st[w], p) for x, w in (("q", "wq"), ("xk", "wk")))
    k, v, page = st["k"].double(), st["v"].double(), st["page"]
    held, new = _grown(case)
    p = torch.cat([torch.arange(a, a + b, device=_DEV) for a, b in zip(held, new)])
    kn, t = _exact_heads(case, st["xk"], st["wk"], p.double()), 0
    table = st["table"].tolist()
    for s, (a, b) in enumerate(zip(held, new)):
        at = torch.tensor(table[s], device=_DEV)[p[t:t + b] // page]
        for h in range(case["kv_heads"]):
            k[0, at, h, p[t:t + b] % page] = kn[t:t + b, h]
            v[0, at, h, p[t:t + b] % page] = st["xv"][t:t + b, h].double()
        t += b
    return [_exact_heads(case, st["q"], st["wq"], p.double()), k, v]


def _exact_heads(case, x, weight, positions):
    """Each pair as a complex number, turned by e^(i angle)."""
    y, R, L = x.double(), case["rot"], case["original"]
    if weight is not None:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / case["dim"] + _EPS) * weight.double()
    f = []
    for p in range(R // 2):
        base = case["base"] * (case["factor"] ** (R / (R - 2)) if case["scaling"] == "base" else 1.0)
        w = math.exp(-2 * p / R * math.log(base))
        if case["scaling"] == "linear":
            w /= case["factor"]
        elif case["scaling"] == "turns":
            n = L * w / math.tau
            w *= 1.0 if n >= 4 else 1 / case["factor"] if n <= 1 else (n - 1) / 3 + (4 - n) / (3 * case["factor"])
        elif case["scaling"] == "pairs":
            first = max(0, math.floor(R / 2 * math.log(L / (32 * math.tau), base)))
            last = min(R - 1, math.ceil(R / 2 * math.log(L / math.tau, base)))
            kept = 1.0 if p <= first else 0.0 if p >= last else (last - p) / (last - first)
            w *= kept + (1 - kept) / case["factor"]
        f.append(w)
    size = 1 + math.log(case["factor"]) / 10 if case["scaling"] == "pairs" else 1.0
    turn = torch.polar(torch.full_like(positions, size)[:, None].expand(-1, R // 2).contiguous(),
                       positions[:, None] * torch.tensor(f, dtype=torch.float64, device=_DEV))[:, None]
    out = y.clone()
    if case["layout"] == "half":
        z = torch.complex(y[..., :R // 2].contiguous(), y[..., R // 2:R].contiguous()) * turn
        out[..., :R // 2], out[..., R // 2:R] = z.real, z.imag
    else:
        z = torch.complex(y[..., 0:R:2].contiguous(), y[..., 1:R:2].contiguous()) * turn
        out[..., 0:R:2], out[..., 1:R:2] = z.real, z.imag
    return out


def _exact_chunk(st):
    q = st["q"]
    out, G, t0 = torch.zeros(q.shape, dtype=torch.float64, device=_DEV), q.shape[1] // st["k"].shape[2], 0
    table, lens, o = st["table"].tolist(), st["lens"].tolist(), st["offsets"].tolist()
    for i, s in enumerate(st["slots"].tolist()):
        t0, nq, n = o[i], o[i + 1] - o[i], lens[s]
        at = torch.tensor(table[s][:_up(n, st["page"])], device=_DEV)
        for h in range(st["k"].shape[2]):
            k, v = (st[x][0, at, h].reshape(-1, q.shape[2])[:n].double() for x in "kv")
            for r in range(0, nq, 1024):
                e = min(nq, r + 1024)
                x = q[t0 + r:t0 + e, h * G:(h + 1) * G].double()
                w = torch.einsum("rgd,nd->rgn", x, k).mul_(st["scale"])
                last = torch.arange(n - nq + r, n - nq + e, device=_DEV)
                w.masked_fill_((torch.arange(n, device=_DEV)[None] > last[:, None])[:, None], -math.inf)
                out[t0 + r:t0 + e, h * G:(h + 1) * G] = torch.softmax(w, -1) @ v
    return out
