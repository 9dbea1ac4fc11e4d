"""The attention and key/value-cache operators, as they are called in a decoder block around the MoE layer, and
their plain forms in elementary torch operations.

prompt   causal attention over packed prompts with grouped heads (Attention.prompt)
decode   one token for each sequence of a batch that shares a long prefix, paged cache (Attention.decode)
write    slots grown and new keys / values written to their pages (KVCache.resize, KVCache.write)
fork     samples of one sequence that share its full pages (KVCache.fork)
compact  live pages moved together (KVCache.compact)

Pool: k, v [layers][pages][kv_heads][page][dim]; table [slots][width] (page of each stretch of a slot's
positions, -1 past its end), lens [slots], refs [pages] (a page is free when its count is 0).
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_DEV = "cuda"


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # the smallest call: a tiny fp32 layer's 64 tokens in five prompts, where launch latency counts
        dict(name="prompt_f32", op="prompt", tokens=64, seqs=5, past=0, heads=4, kv_heads=2, dim=32, dtype="f32", pick=1),
        # an ordinary prefill batch at d = 4096 (32 heads of 128): prompts of very different lengths, packed
        dict(name="prompt_ragged", op="prompt", tokens=8192, seqs=13, past=0, heads=32, kv_heads=8, dim=128, dtype="bf16",
             pick=2),
        # the largest prefill: one prompt of 16384 tokens at d = 4096
        dict(name="prompt_long", op="prompt", tokens=16384, seqs=1, past=0, heads=32, kv_heads=8, dim=128, dtype="bf16",
             pick=3),
        # one conversation, one token: nothing shared, d = 8192 (64 heads of 128)
        dict(name="decode_t1", op="decode", seqs=1, shared=0, own=4096, heads=64, kv_heads=8, dim=128, page=64, dtype="bf16",
             pick=4),
        # eight samples of one prompt of 8192 tokens
        dict(name="decode_t8", op="decode", seqs=8, shared=8192, own=512, heads=64, kv_heads=8, dim=128, page=64,
             dtype="bf16", pick=5),
        # a serving batch of 64 behind one system prompt of 32768 tokens
        dict(name="decode_t64", op="decode", seqs=64, shared=32768, own=2048, heads=64, kv_heads=8, dim=128, page=64,
             dtype="bf16", pick=6),
        # a decode step's new token of 64 sequences
        dict(name="write_step", op="write", seqs=64, base=2048, new=64, kv_heads=8, dim=128, page=64, dtype="bf16", pick=7),
        # eight prompts admitted together
        dict(name="write_prompt", op="write", seqs=8, base=0, new=16384, kv_heads=8, dim=128, page=64, dtype="bf16", pick=8),
        # a beam search's step: 16 dropped beams take over 16 kept ones; four layers
        dict(name="fork_beams", op="fork", seqs=16, fan=1, length=1500, layers=4, kv_heads=8, dim=128, page=16, dtype="bf16",
             pick=9),
        # 64 samples started from one prompt of about 16 thousand tokens; eight layers
        dict(name="fork_samples", op="fork", seqs=1, fan=64, length=16000, layers=8, kv_heads=8, dim=128, page=64,
             dtype="bf16", pick=10),
        # a small pool with holes
        dict(name="compact_small", op="compact", pages=300, live=0.4, layers=1, kv_heads=2, dim=64, page=16, dtype="bf16",
             pick=11),
        # a large pool after a burst of finished requests: about 900 pages of 256 KB to move
        dict(name="compact_large", op="compact", pages=4000, live=0.35, layers=1, kv_heads=8, dim=128, page=64,
             dtype="bf16", pick=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "decode", "decode", "decode", "write", "fork", "compact"])
    c = dict(op=op, pick=rng.randrange(1 << 20))
    kv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([g for g in (1, 2, 3, 4, 6, 8) if g * kv <= (32 if op == "prompt" else 64)])
    dim = rng.choice([64, 64, 128, 128, 128, 32, 80, 96])
    if op == "prompt":
        f32 = rng.random() < 0.2
        tokens = _log_int(rng, 1, 1024 if f32 else 12000)
        c.update(tokens=tokens, seqs=min(tokens, _log_int(rng, 1, 40)), past=rng.choice([0, 0, _log_int(rng, 1, 2000)]),
                 heads=kv * group, kv_heads=kv, dim=dim, dtype="f32" if f32 else "bf16")
        return c
    page = rng.choice([16, 32, 64, 128])
    if op == "decode":
        f32 = rng.random() < 0.2
        shared = rng.choice([0, _log_int(rng, page, 4096 if f32 else 32768)]) // page * page
        c.update(seqs=_log_int(rng, 1, 64), shared=shared, own=_log_int(rng, 1, 512 if f32 else 4096), heads=kv * group,
                 kv_heads=kv, dim=dim, page=page, dtype="f32" if f32 else "bf16")
        return c
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "write":
        n = _log_int(rng, 1, 64)
        c.update(seqs=n, base=rng.choice([0, _log_int(rng, 1, 2048)]), new=n * _log_int(rng, 1, 128) + rng.randrange(n),
                 kv_heads=kv, dim=dim, page=page, dtype=dtype)
    elif op == "fork":
        c.update(seqs=_log_int(rng, 1, 8), fan=_log_int(rng, 1, 8), length=_log_int(rng, 1, 4096), layers=rng.choice([1, 2, 4]),
                 kv_heads=kv, dim=dim, page=page, dtype=dtype)
    else:
        c.update(pages=_log_int(rng, 8, 2000), live=round(rng.uniform(0.1, 0.9), 3), layers=rng.choice([1, 2]), kv_heads=kv,
                 dim=dim, page=page, dtype=dtype)
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


def _ragged(case):
    """Query lengths and key lengths of a prompt case."""
    nq = _parts(case["tokens"], case["seqs"], case["pick"])
    r = random.Random(case["pick"] + 1)
    return nq, [a + (r.randint(0, case["past"]) if case["past"] else 0) for a in nq]


def _own_lens(case):
    """Keys of a decode case's sequences after the shared ones; the first has as many as any may have."""
    r = random.Random(case["pick"])
    return [case["own"]] + [r.randint(0 if case["shared"] else 1, case["own"]) for _ in range(case["seqs"] - 1)]


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


def _pool(g, case, layers, pages):
    shape = (layers, pages, case["kv_heads"], case["page"], case["dim"])
    t = _TYPES[case["dtype"]]
    k = torch.empty(shape, dtype=t, device=_DEV)
    v = torch.empty(shape, dtype=t, device=_DEV)
    for x in (k, v):
        for layer in range(layers):
            x[layer].copy_(torch.randn(shape[1:], generator=g, device=_DEV, dtype=torch.float32))
    v += 0.5 * torch.randn((case["dim"],), generator=g, device=_DEV).to(t)
    return k, v


def _table(rows, width):
    return _ints([r + [-1] * (width - len(r)) for r in rows])


def _counts(rows, pages):
    n = [0] * pages
    for r in rows:
        for p in r:
            n[p] += 1
    return _ints(n)


def _cache_state(case, g, rows, lens, pages, width, layers=1):
    k, v = _pool(g, case, layers, pages)
    st = dict(k=k, v=v, table=_table(rows, width), lens=_ints(lens), refs=_counts(rows, pages), page=case["page"])
    if own:  # the handle that a user's program keeps for its cache
        import sparse_mixture_experts_moe_gb300 as moe
        st["cache"] = moe.KVCache(st["k"], st["v"], st["table"], st["lens"], st["refs"])
    return st


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    r = random.Random(seed)
    if op == "prompt":
        nq, nk = _ragged(case)
        H, Hk, D, t = case["heads"], case["kv_heads"], case["dim"], _TYPES[case["dtype"]]
        shift = 0.5 * torch.randn((D,), generator=g, device=_DEV)
        if case["past"] == 0:  # q, k and v as slices of one fused projection of the tokens
            x = torch.randn((sum(nq), H + 2 * Hk, D), generator=g, device=_DEV)
            x[:, H + Hk:] += shift
            x = x.to(t)
            q, k, v = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
        else:
            q = _normal(g, (sum(nq), H, D), t)
            k = _normal(g, (sum(nk), Hk, D), t)
            v = (torch.randn((sum(nk), Hk, D), generator=g, device=_DEV) + shift).to(t)
        st = dict(op=op, q=q, k=k, v=v, qo=_ints(_offsets(nq)), ko=_ints(_offsets(nk)), lq=max(nq), lk=max(nk),
                  scale=D ** -0.5)
    elif op == "decode":
        S, page, H, D = case["shared"], case["page"], case["heads"], case["dim"]
        lens = [S + a for a in _own_lens(case)]
        need = [_up(a, page) - S // page for a in lens]
        pages = S // page + sum(need) + 5
        order = list(range(pages))
        r.shuffle(order)  # pages as churn leaves them
        head, at, rows = order[:S // page], S // page, []
        for a in need:
            rows.append(head + order[at:at + a])
            at += a
        st = _cache_state(case, g, rows, lens, pages, _up(S + case["own"], page) + 1)
        x = _normal(g, (case["seqs"], H + 2 * case["kv_heads"], D), _TYPES[case["dtype"]])
        st.update(op=op, q=x[:, :H], slots=_ints(list(range(case["seqs"]))), shared=S, most=max(lens), scale=D ** -0.5)
    elif op == "write":
        page, n = case["page"], case["seqs"]
        base = _base_lens(case)
        new = _parts(case["new"], n, case["pick"])
        pages = sum(_up(a + b, page) for a, b in zip(base, new)) + 7
        order = list(range(pages))
        r.shuffle(order)
        rows, at = [], 0
        for a in base:
            rows.append(order[at:at + _up(a, page)])
            at += _up(a, page)
        st = _cache_state(case, g, rows, base, pages, _up(max(a + b for a, b in zip(base, new)), page) + 1)
        t = _TYPES[case["dtype"]]
        x = _normal(g, (sum(new), 2 * case["kv_heads"], case["dim"]), t)
        st.update(op=op, xk=x[:, :case["kv_heads"]], xv=x[:, case["kv_heads"]:], slots=_ints(list(range(n))),
                  base=_ints(base), grown=_ints([a + b for a, b in zip(base, new)]), offsets=_ints(_offsets(new)))
    elif op == "fork":
        page, n, m = case["page"], case["seqs"], case["seqs"] * case["fan"]
        rows, lens, at, pages, order = [], [], 0, *_fork_pages(case, r)
        for a in _fork_lens(case):
            rows.append(order[at:at + _up(a, page)])
            lens.append(a)
            at += _up(a, page)
        st = _cache_state(case, g, rows, lens, pages, _up(case["length"], page) + 1, case["layers"])
        st.update(op=op, src=_ints([i % n for i in range(m)]), dst=_ints([n + i for i in range(m)]))
    else:
        page, pages = case["page"], case["pages"]
        rows, lens = _holes(case, r)
        st = _cache_state(case, g, rows, lens, pages, max(len(x) for x in rows) + 1, case["layers"])
        st.update(op=op, table0=st["table"].clone(), refs0=st["refs"].clone())
    if own and op in ("prompt", "decode"):
        import sparse_mixture_experts_moe_gb300 as moe
        st["attention"] = moe.Attention(case["heads"], case["kv_heads"], case["dim"], _TYPES[case["dtype"]])
    return st


def _base_lens(case):
    r = random.Random(case["pick"])
    return [r.randint(0, case["base"]) for _ in range(case["seqs"])]


def _fork_lens(case):
    """Lengths of the kept sequences, then of what the slots taken over held before."""
    r = random.Random(case["pick"])
    n, m = case["seqs"], case["seqs"] * case["fan"]
    kept = [r.randint(max(1, case["length"] // 2), case["length"]) for _ in range(n)]
    return kept + [r.randint(0, case["length"]) if case["fan"] == 1 else 0 for _ in range(m)]


def _fork_pages(case, r):
    pages = sum(_up(a, case["page"]) for a in _fork_lens(case)) + case["seqs"] * case["fan"] + 9
    order = list(range(pages))
    r.shuffle(order)
    return pages, order


def _holes(case, r):
    """Slots whose pages lie anywhere in a pool of which the share `live` is in use; every third slot shares its
    first page with the one before."""
    pages, page, shape = case["pages"], case["page"], random.Random(case["pick"])
    order = list(range(pages))
    r.shuffle(order)
    left, rows, lens = order[:max(1, int(pages * case["live"]))], [], []
    while left:
        a = min(len(left), shape.randint(1, 40))
        row, left = left[:a], left[a:]
        if len(rows) % 3 == 2:
            row = rows[-1][:1] + row
        rows.append(row)
        lens.append(len(row) * page - shape.randrange(page))
    return rows, lens


# ---------------------------------------------------------------------------------------------- one pass

def run(st):
    return _OWN[st["op"]](st) if own else _PLAIN[st["op"]](st)


def _pools(st, *more):
    return [st["k"], st["v"], st["table"], st["lens"], st["refs"], *more]


def _own_prompt(st):
    return st["attention"].prompt(st["q"], st["k"], st["v"], st["qo"], st["ko"])


def _own_decode(st):
    return st["attention"].decode(st["q"], st["cache"], st["slots"], shared_len=st["shared"])


def _own_write(st):
    c = st["cache"]
    c.resize(st["slots"], st["base"])  # drafted tokens of the last pass rolled back
    c.resize(st["slots"], st["grown"])
    c.write(st["xk"], st["xv"], st["slots"], st["offsets"], st["base"])
    return _pools(st)


def _own_fork(st):
    st["cache"].fork(st["src"], st["dst"])
    return _pools(st)


def _own_compact(st):
    st["table"].copy_(st["table0"])  # the tables as churn left them
    st["refs"].copy_(st["refs0"])
    return _pools(st, st["cache"].compact())


_OWN = {"prompt": _own_prompt, "decode": _own_decode, "write": _own_write, "fork": _own_fork, "compact": _own_compact}


def _plain_prompt(st):
    qo, ko, lq, lk = st["qo"].long(), st["ko"].long(), st["lq"], st["lk"]
    n, (T, H, D), Hk = qo.numel() - 1, st["q"].shape, st["k"].shape[1]
    G = H // Hk
    i, j = torch.arange(lq, device=_DEV), torch.arange(lk, device=_DEV)
    nq, nk = qo[1:] - qo[:-1], ko[1:] - ko[:-1]
    q = st["q"].float()[(qo[:-1, None] + i).clamp(max=T - 1)]                       # [n, lq, H, D], padded
    rows = (ko[:-1, None] + j).clamp(max=st["k"].shape[0] - 1)
    k, v = st["k"].float()[rows].transpose(1, 2), st["v"].float()[rows].transpose(1, 2)  # [n, Hk, lk, D]
    q = q.view(n, lq, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(n, Hk, G * lq, D) * st["scale"]
    s = (q @ k.transpose(2, 3)).view(n, Hk, G, lq, lk)
    hidden = j > (i[:, None] + (nk - nq)[:, None, None])                             # [n, lq, lk]
    s.masked_fill_(hidden[:, None, None], float("-inf"))
    s -= s.amax(-1, keepdim=True)
    s.exp_()
    o = (s.view(n, Hk, G * lq, lk) @ v).view(n, Hk, G, lq, D) / s.sum(-1, keepdim=True)
    t = torch.arange(T, device=_DEV)
    seq = (t[:, None] >= qo[None, 1:]).sum(1)
    return o[seq, :, :, t - qo[seq]].reshape(T, H, D).to(st["q"].dtype)


def _plain_decode(st):
    page, S, (n, H, D), Hk = st["page"], st["shared"], st["q"].shape, st["k"].shape[2]
    G, P = H // Hk, S // page
    slots = st["slots"].long()
    rows, lens = st["table"][slots].long(), st["lens"][slots]
    most = _up(st["most"], page)
    q = st["q"].float().view(n, Hk, G, D) * st["scale"]
    # the shared keys, once for all rows
    kp = st["k"][0, rows[0, :P]].float().transpose(0, 1).reshape(Hk, S, D)
    vp = st["v"][0, rows[0, :P]].float().transpose(0, 1).reshape(Hk, S, D)
    qs = q.transpose(0, 1).reshape(Hk, n * G, D)
    a = (qs @ kp.transpose(1, 2)).view(Hk, n, G, S).transpose(0, 1)                  # [n, Hk, G, S]
    # each sequence's own keys, padded
    at = rows[:, P:most].clamp(min=0)
    L = at.shape[1] * page
    ko = st["k"][0, at].float().transpose(1, 2).reshape(n, Hk, L, D)
    vo = st["v"][0, at].float().transpose(1, 2).reshape(n, Hk, L, D)
    b = q @ ko.transpose(2, 3)
    hidden = S + torch.arange(L, device=_DEV) >= lens[:, None]
    b = b.masked_fill(hidden[:, None, None], float("-inf"))
    m = torch.cat([a, b], -1).amax(-1, keepdim=True)
    a, b = torch.exp(a - m), torch.exp(b - m)
    o = (a.transpose(0, 1).reshape(Hk, n * G, S) @ vp).view(Hk, n, G, D).transpose(0, 1) + b @ vo
    return (o / (a.sum(-1, keepdim=True) + b.sum(-1, keepdim=True))).reshape(n, H, D).to(st["q"].dtype)


def _free_first(refs):
    """Page numbers, the free ones first, ascending."""
    return torch.sort((refs != 0).to(torch.int32), stable=True).indices


def _release(st, rows, drop):
    st["refs"].index_add_(0, rows.clamp(min=0).reshape(-1), -drop.reshape(-1).to(torch.int32))


def _copy_pages(st, src, dst):
    st["k"][:, dst] = st["k"][:, src]
    st["v"][:, dst] = st["v"][:, src]


def _plain_resize(st, slots, new):
    page, refs = st["page"], st["refs"]
    slots, new = slots.long(), new.long()
    rows, old = st["table"][slots].long(), st["lens"][slots].long()
    c = torch.arange(rows.shape[1], device=_DEV)
    po, pn = -(-old // page), -(-new // page)
    drop = (c >= pn[:, None]) & (c < po[:, None])
    _release(st, rows, drop)
    rows = torch.where(drop, -1, rows)
    # a partly filled last page that others hold too is copied when its slot grows
    last = rows.gather(1, (po - 1).clamp(min=0)[:, None])[:, 0].clamp(min=0)
    cow = (new > old) & (old % page != 0) & (refs[last] > 1)
    first = po - cow.long()
    need = (pn - first).clamp(min=0)
    start = need.cumsum(0) - need
    free = _free_first(refs)
    take = (c >= first[:, None]) & (c < pn[:, None])
    got = free[(start[:, None] + c - first[:, None]).clamp(0, free.numel() - 1)]
    rows = torch.where(take, got, rows)
    mine = rows.gather(1, (po - 1).clamp(min=0)[:, None])[:, 0]
    _copy_pages(st, last[cow], mine[cow])
    refs.index_add_(0, last, -cow.to(torch.int32))
    refs.index_add_(0, rows.clamp(min=0).reshape(-1), take.reshape(-1).to(torch.int32))
    st["table"][slots] = rows.to(torch.int32)
    st["lens"][slots] = new.to(torch.int32)


def _plain_write(st):
    _plain_resize(st, st["slots"], st["base"])
    _plain_resize(st, st["slots"], st["grown"])
    o = st["offsets"].long()
    t = torch.arange(st["xk"].shape[0], device=_DEV)
    i = (t[:, None] >= o[None, 1:]).sum(1)
    p = st["base"].long()[i] + t - o[i]
    at = st["table"][st["slots"].long()[i], p // st["page"]].long()
    st["k"][0].transpose(1, 2)[at, p % st["page"]] = st["xk"]
    st["v"][0].transpose(1, 2)[at, p % st["page"]] = st["xv"]
    return _pools(st)


def _plain_fork(st):
    page, src, dst = st["page"], st["src"].long(), st["dst"].long()
    c = torch.arange(st["table"].shape[1], device=_DEV)
    rows = st["table"][dst].long()
    _release(st, rows, c < (-(-st["lens"][dst].long() // page))[:, None])
    rows, n = st["table"][src].long(), st["lens"][src].long()
    full, part = n // page, (n % page != 0).long()
    free = _free_first(st["refs"])
    got = free[(part.cumsum(0) - part).clamp(max=free.numel() - 1)]
    tail = rows.gather(1, full.clamp(max=rows.shape[1] - 1)[:, None])[:, 0]
    new = torch.where(c < full[:, None], rows, torch.where((c == full[:, None]) & (part[:, None] == 1), got[:, None], -1))
    _copy_pages(st, tail[part == 1], got[part == 1])
    st["refs"].index_add_(0, new.clamp(min=0).reshape(-1), (new >= 0).reshape(-1).to(torch.int32))
    st["table"][dst] = new.to(torch.int32)
    st["lens"][dst] = n.to(torch.int32)
    return _pools(st)


def _plain_compact(st):
    st["table"].copy_(st["table0"])
    st["refs"].copy_(st["refs0"])
    refs, table = st["refs"], st["table"]
    live, i = refs > 0, torch.arange(refs.numel(), device=_DEV)
    count = live.sum()
    src, dst = (live & (i >= count)).nonzero()[:, 0], (~live & (i < count)).nonzero()[:, 0]
    _copy_pages(st, src, dst)
    to = i.clone()
    to[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].to(torch.int32), -1))
    return _pools(st, count.to(torch.int32).reshape(1))


_PLAIN = {"prompt": _plain_prompt, "decode": _plain_decode, "write": _plain_write, "fork": _plain_fork,
          "compact": _plain_compact}


# ---------------------------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, eb, D = case["op"], 4 if case["dtype"] == "f32" else 2, case["dim"]
    kv = 2 * case["kv_heads"] * D * eb  # K and V of one position
    if op == "prompt":
        nq, nk = _ragged(case)
        pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(nq, nk))
        return {"bytes": 2 * sum(nq) * case["heads"] * D * eb + sum(nk) * kv, "flops": 4 * D * case["heads"] * pairs}
    if op == "decode":
        lens = _own_lens(case)
        return {"bytes": (case["shared"] + sum(lens)) * kv + 2 * case["seqs"] * case["heads"] * D * eb,
                "flops": 4 * D * case["heads"] * (case["seqs"] * case["shared"] + sum(lens))}
    if op == "write":
        new = _parts(case["new"], case["seqs"], case["pick"])
        return {"bytes": 2 * sum(new) * kv + 8 * sum(_up(a, case["page"]) for a in new), "flops": 0}
    one = 2 * case["layers"] * case["page"] * kv  # a page read and written
    if op == "fork":
        lens = _fork_lens(case)[:case["seqs"]]
        part = sum(a % case["page"] != 0 for a in lens) * case["fan"]
        return {"bytes": part * one + case["fan"] * sum(_up(a, case["page"]) for a in lens) * 12, "flops": 0}
    rows, _ = _holes(case, random.Random(case["pick"]))
    live = {p for x in rows for p in x}
    return {"bytes": sum(p >= len(live) for p in live) * one + 8 * (sum(map(len, rows)) + case["pages"]), "flops": 0}


# ---------------------------------------------------------------------------------------------- from the definitions, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "prompt":
        return _exact_prompt(st, *_ragged(case))
    if case["op"] == "decode":
        return _exact_decode(st)
    return _exact_cache(st, case)


def _attend(q, k, v, see, scale):
    """Rows q [r, D] over keys k, v [n, D]; see [r]: how many of the first keys each row sees."""
    w = torch.einsum("rd,nd->rn", q, k).mul_(scale)
    w[torch.arange(k.shape[0], device=_DEV)[None, :] >= see[:, None]] = -math.inf
    return torch.softmax(w, 1) @ v


def _exact_prompt(st, nq, nk):
    q, k, v = (st[x].double() for x in "qkv")
    out, G = torch.zeros_like(q), q.shape[1] // k.shape[1]
    q0 = k0 = 0
    for a, b in zip(nq, nk):
        for h in range(q.shape[1]):
            for r in range(0, a, 2048):
                see = torch.arange(r, min(a, r + 2048), device=_DEV) + 1 + b - a
                n = min(a, r + 2048) + b - a
                out[q0 + r:q0 + min(a, r + 2048), h] = _attend(q[q0 + r:q0 + min(a, r + 2048), h], k[k0:k0 + n, h // G],
                                                              v[k0:k0 + n, h // G], see, st["scale"])
        q0, k0 = q0 + a, k0 + b
    return out


def _exact_decode(st):
    q = st["q"].double()
    n, H, D = q.shape
    out, G = torch.zeros_like(q), H // st["k"].shape[2]
    table, lens = st["table"].tolist(), st["lens"].tolist()
    for i, s in enumerate(st["slots"].tolist()):
        at = torch.tensor(table[s][:_up(lens[s], st["page"])], device=_DEV)
        for h in range(H // G):
            k, v = (st[x][0, at, h].reshape(-1, D)[:lens[s]].double() for x in "kv")
            see = torch.full((G,), lens[s], device=_DEV)
            out[i, h * G:(h + 1) * G] = _attend(q[i, h * G:(h + 1) * G], k, v, see, st["scale"])
    return out


def _exact_cache(st, case):
    """The bookkeeping on lists, page by page, and the pages as they end up."""
    page, k, v = case["page"], st["k"].double(), st["v"].double()
    rows = [[p for p in r if p >= 0] for r in st["table"].tolist()]
    lens, refs, width = st["lens"].tolist(), st["refs"].tolist(), st["table"].shape[1]
    low = 0  # no page below this one is free

    def new_page():
        nonlocal low
        low = refs.index(0, low)
        refs[low] = 1
        return low

    def copy(a, b):
        k[:, b] = k[:, a]
        v[:, b] = v[:, a]

    more = []
    if case["op"] == "write":
        base, grown, o = st["base"].tolist(), st["grown"].tolist(), st["offsets"].tolist()
        for i, s in enumerate(st["slots"].tolist()):
            for _ in range(_up(grown[i], page) - len(rows[s])):
                rows[s].append(new_page())
            lens[s] = grown[i]
            p = torch.arange(base[i], grown[i], device=_DEV)
            at = torch.tensor(rows[s] + [0], device=_DEV)[p // page]
            k[0].transpose(1, 2)[at, p % page] = st["xk"][o[i]:o[i + 1]].double()
            v[0].transpose(1, 2)[at, p % page] = st["xv"][o[i]:o[i + 1]].double()
    elif case["op"] == "fork":
        src, dst = st["src"].tolist(), st["dst"].tolist()
        for d in dst:
            for p in rows[d]:
                refs[p] -= 1
            rows[d] = []
        for s, d in zip(src, dst):
            full = lens[s] // page
            rows[d], lens[d] = rows[s][:full], lens[s]
            for p in rows[d]:
                refs[p] += 1
            if lens[s] % page:
                rows[d].append(new_page())
                copy(rows[s][full], rows[d][full])
    else:
        count = sum(c > 0 for c in refs)
        holes = [p for p in range(count) if refs[p] == 0]
        moved = {}
        for p in range(count, len(refs)):
            if refs[p]:
                moved[p] = holes.pop(0)
                copy(p, moved[p])
                refs[moved[p]], refs[p] = refs[p], 0
        rows = [[moved.get(p, p) for p in r] for r in rows]
        more = [_ints([count])]
    return [k, v, _table(rows, width), _ints(lens), _ints(refs), *more]
