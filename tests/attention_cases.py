"""Inputs, fp64 references and error bounds of the attention and cache tests.

A floating output is held to a bound per element that counts its roundings. With p the softmax weights and
a half step of h(t) = finfo(t).eps / 2 relative to a value of type t:
  out         h(dt) |ref|                        the one rounding of the result
  weights     h(bf16) sum p |v|  (bf16 only)     a weight may be rounded to bf16 before it meets v
  scores      2 d sum p |v|                      d: the largest absolute error of a score, which moves a weight by
                                                 the factor e^d and the sum by no more;
                                                 d = (D + 8) h(fp32) max_j scale sum |q k_j| + 2^-21 (the power of two)
  sums        2 (n + 64) h(fp32) sum p |v|       n keys added in fp32, above and below the fraction, in any
                                                 order and any number of parts
"""
from __future__ import annotations

import random

import numpy as np
import torch

H32 = 2.0 ** -24
H16 = 2.0 ** -8


def tensor(shape, seed, dtype, device, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(dtype).to(device)


def attend64(q, k, v, limits, scale):
    """out [H, r, D], lse [H, r] and the weights' sum of |v| and largest absolute score sums, in fp64 on the host.
    q [r, H, D], k, v [n, Hk, D]; limits [r]: how many first keys each row sees."""
    r, H, D = q.shape
    n, Hk, _ = k.shape
    G = H // Hk
    out = np.zeros((r, H, D))
    lse = np.full((r, H), -np.inf)
    pv = np.zeros((r, H, D))
    big = np.zeros((r, H))
    for h in range(H):
        kk, vv = k[:, h // G], v[:, h // G]
        for i in range(r):
            m = int(limits[i])
            if m <= 0:
                continue
            s = scale * (kk[:m] @ q[i, h])
            top = s.max()
            w = np.exp(s - top)
            z = w.sum()
            w /= z
            out[i, h] = w @ vv[:m]
            pv[i, h] = w @ np.abs(vv[:m])
            lse[i, h] = top + np.log(z)
            big[i, h] = scale * (np.abs(kk[:m]) @ np.abs(q[i, h])).max()
    return out, lse, pv, big


def bounds(out, pv, big, n, D, dtype):
    """(bound per output element, bound per lse entry)."""
    d = (D + 8) * H32 * big + 2.0 ** -21
    rel = 2 * d + 2 * (n + 64) * H32
    if dtype == torch.bfloat16:
        o = H16 * np.abs(out) + (H16 + rel)[..., None] * pv * (1 + H16)
    else:
        o = H32 * np.abs(out) + rel[..., None] * pv
    return o + 1e-30, d + 2 * (n + 64) * H32 + 2.0 ** -20


def check(got, lse, ref, n, D, dtype):
    out, l64, pv, big = ref
    g = got.detach().to(torch.float64).cpu().numpy()
    bo, bl = bounds(out, pv, big, n, D, dtype)
    err = np.abs(g - out)
    assert np.isfinite(g).all()
    assert (err <= bo).all(), f"out off by {float((err / bo).max()):.3g} times its bound"
    if lse is not None:
        l = lse.detach().to(torch.float64).cpu().numpy()
        empty = np.isneginf(l64)
        assert (np.isneginf(l) == empty).all()
        e = np.abs(np.where(empty, 0, l) - np.where(empty, 0, l64))
        assert (e <= bl).all(), f"lse off by {float((e / bl).max()):.3g} times its bound"


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def prompt_reference(q, k, v, qo, ko, causal, scale):
    T, H, D = q.shape
    out, lse, pv, big = np.zeros((T, H, D)), np.full((T, H), -np.inf), np.zeros((T, H, D)), np.zeros((T, H))
    for i in range(len(qo) - 1):
        a, b, nq, nk = qo[i], ko[i], qo[i + 1] - qo[i], ko[i + 1] - ko[i]
        if nq == 0:
            continue
        lim = [max(0, min(nk, t + 1 + nk - nq)) if causal else nk for t in range(nq)]
        r = attend64(f64(q[a:a + nq]), f64(k[b:b + nk]), f64(v[b:b + nk]), lim, scale)
        out[a:a + nq], lse[a:a + nq], pv[a:a + nq], big[a:a + nq] = r
    return out, lse, pv, big


def offsets(lens):
    return [0] + np.cumsum(lens).tolist()


def i32(v, device):
    return torch.tensor(v, dtype=torch.int32, device=device)


class Model:
    """A cache's tables on plain lists: what every cache call must leave behind, page by page."""

    def __init__(self, n_layers, n_pages, page, n_slots, width):
        self.layers, self.page, self.width = n_layers, page, width
        self.rows = [[] for _ in range(n_slots)]
        self.lens = [0] * n_slots
        self.refs = [0] * n_pages
        self.k = self.v = None  # torch tensors on the host

    def up(self, n):
        return -(-n // self.page)

    def _free(self, want):
        f = [p for p, r in enumerate(self.refs) if r == 0]
        return f[:want]

    def _copy(self, a, b):
        self.k[:, b] = self.k[:, a]
        self.v[:, b] = self.v[:, a]

    def resize(self, slots, lens):
        """Returns the entries that were skipped."""
        bad, todo = [], []
        seen = set()
        for i, (s, n) in enumerate(zip(slots, lens)):
            if not 0 <= s < len(self.rows) or not 0 <= n <= self.width * self.page or s in seen:
                bad.append(i)
                continue
            seen.add(s)
            todo.append((i, s, n))
        for _, s, n in todo:
            while len(self.rows[s]) > self.up(n):
                self.refs[self.rows[s].pop()] -= 1
        need = []
        for i, s, n in todo:
            cow = n > self.lens[s] and self.lens[s] % self.page != 0 and self.refs[self.rows[s][-1]] > 1
            need.append((i, s, n, cow, max(0, self.up(n) - len(self.rows[s])) + cow))
        free = self._free(sum(x[4] for x in need))
        at = 0
        copies = []
        for i, s, n, cow, want in need:
            got = free[at:at + want]
            at += want
            if len(got) < want:
                bad.append(i)
                continue
            if cow:
                old = self.rows[s].pop()
                copies.append((old, got[0]))
                self.refs[old] -= 1
            self.rows[s] += got
            for p in got:
                self.refs[p] = 1
            self.lens[s] = n
        for a, b in copies:
            self._copy(a, b)
        return bad

    def fork(self, src, dst):
        bad, todo, seen = [], [], set()
        n = len(self.rows)
        sources = {s for s, d in zip(src, dst) if 0 <= s < n and 0 <= d < n}
        for i, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < n and 0 <= d < n) or d in seen or d in sources:
                bad.append(i)
                if 0 <= s < n and 0 <= d < n:
                    seen.add(d)
                continue
            seen.add(d)
            todo.append((i, s, d))
        for _, s, d in todo:
            for p in self.rows[d]:
                self.refs[p] -= 1
            self.rows[d], self.lens[d] = [], 0
        part = [self.lens[s] % self.page != 0 for _, s, _ in todo]
        free, at = self._free(sum(part)), 0
        for (i, s, d), t in zip(todo, part):
            full = self.lens[s] // self.page
            if t and at >= len(free):
                bad.append(i)
                at += 1
                continue
            self.rows[d] = self.rows[s][:full]
            for p in self.rows[d]:
                self.refs[p] += 1
            if t:
                self._copy(self.rows[s][full], free[at])
                self.rows[d].append(free[at])
                self.refs[free[at]] = 1
                at += 1
            self.lens[d] = self.lens[s]
        return bad

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        holes = [p for p in range(live) if self.refs[p] == 0]
        move = {}
        for p in range(live, len(self.refs)):
            if self.refs[p]:
                move[p] = holes.pop(0)
        for a, b in move.items():
            self._copy(a, b)
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.rows = [[move.get(p, p) for p in r] for r in self.rows]
        return live

    def write(self, layer, slots, offs, pos, k, v):
        for i, s in enumerate(slots):
            for t in range(offs[i], offs[i + 1]):
                p = pos[i] + t - offs[i]
                page = self.rows[s][p // self.page]
                self.k[layer, page, :, p % self.page] = k[t]
                self.v[layer, page, :, p % self.page] = v[t]

    def table(self):
        return [r + [-1] * (self.width - len(r)) for r in self.rows]

    def keys(self, layer, slot):
        """K and V of a slot, [len, Hk, D] in fp64."""
        n = self.lens[slot]
        if n == 0:
            z = np.zeros((0, self.k.shape[2], self.k.shape[4]))
            return z, z
        at = torch.tensor(self.rows[slot])
        return tuple(f64(x[layer, at].transpose(1, 2).reshape(-1, x.shape[2], x.shape[4])[:n]) for x in (self.k, self.v))


def random_lens(rng: random.Random, n, most, zero=0.15):
    return [0 if rng.random() < zero else rng.randint(1, most) for _ in range(n)]
