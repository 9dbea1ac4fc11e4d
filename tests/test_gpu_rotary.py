"""Rotary positions, norms of heads and appending to the paged cache against the formulas in fp64.

Bounds per element, with h(t) = finfo(t).eps / 2 and c, s the cosine and sine times the magnitude: a result is
y_a c - y_b s with y = x inv w (y = x without a norm). In fp32 the products and sums, the mean (D terms), the reciprocal
square root (2 ulp), the weight, and cosine and sine (within 2^-22 of the magnitude: the angle's 2^-32 of a circle, its
conversion and the polynomials' roundings) move it by at most (D + 32) h(fp32) |y_a| + |y_b| times the magnitude; rounding
to the type adds h(t) of the result.
"""
import math
import random

import numpy as np
import pytest
import torch

import sparse_mixture_experts_moe_gb300 as moe
from attention_cases import H32, Model, f64, i32, offsets, tensor

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def turned64(x, positions, rope, base, weight=None, eps=1e-6, magnitude=1.0, frequencies=None):
    """(result, bound without the last rounding) of x [T, H, D] in fp64."""
    y = f64(x)
    D, R = rope.head_dim, rope.rotary_dim
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * f64(weight)
    f = np.array(frequencies if frequencies is not None else [base ** (-2 * p / R) for p in range(R // 2)])
    a = np.asarray(positions, dtype=np.float64)[:, None, None] * f
    c, s = np.cos(a) * magnitude, np.sin(a) * magnitude
    out, far = y.copy(), np.abs(y)
    if rope.layout == "half":
        i, j = slice(0, R // 2), slice(R // 2, R)
    else:
        i, j = slice(0, R, 2), slice(1, R, 2)
    out[..., i], out[..., j] = y[..., i] * c - y[..., j] * s, y[..., j] * c + y[..., i] * s
    far[..., i] = far[..., j] = (np.abs(y[..., i]) + np.abs(y[..., j])) * abs(magnitude)
    return out, (D + 32) * H32 * far


def close(got, ref, dtype):
    want, bound = ref
    err = np.abs(f64(got) - want)
    bound = bound + torch.finfo(dtype).eps / 2 * (np.abs(want) + bound) + 1e-37
    assert (err <= bound).all(), f"off by {float((err / bound).max()):.3g} times the bound"


SHAPES = [(64, 64), (128, 128), (128, 64), (80, 80), (80, 20), (80, 40), (96, 24), (256, 256), (256, 64), (8, 8), (8, 2), (8, 4),
          (24, 6), (136, 136), (248, 16), (200, 26), (64, 0), (16, 14), (32, 30)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,R", SHAPES)
@pytest.mark.parametrize("norm", [False, True])
def test_apply_heads(D, R, layout, norm, dtype):
    r = random.Random(D * 1000 + R)
    T, H, Hk = 37, 6, 3
    x = tensor((T, H + 2 * Hk, D), D + R, dtype, DEV)  # slices of one projection
    q, k = x[:, :H], x[:, H:H + Hk]
    pos = [r.choice([0, 1, 7, r.randrange(5000), r.randrange(1 << 20)]) for _ in range(T)]
    wq, wk = (tensor((D,), s, dtype, DEV) if norm else None for s in (1, 2))
    rope = moe.Rotary(D, rotary_dim=R, layout=layout)
    a, b = rope.apply(q, i32(pos, DEV), k, q_weight=wq, k_weight=wk)
    close(a, turned64(q, pos, rope, 1e4, wq), dtype)
    close(b, turned64(k, pos, rope, 1e4, wk), dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H,Hk", [(1, 1, 1), (1, 64, 8), (2, 3, 0), (7, 40, 8), (65, 5, 5), (3000, 2, 1), (5000, 9, 0), (9, 300, 1)])
def test_apply_sizes(T, H, Hk, dtype):
    rope = moe.Rotary(64, base=5e5)
    q = tensor((T, H, 64), T, dtype, DEV)
    k = tensor((T, Hk, 64), T + 1, dtype, DEV) if Hk else None
    pos = list(range(100, 100 + T))
    w = tensor((64,), 3, dtype, DEV)
    got = rope.apply(q, i32(pos, DEV), k, q_weight=w)
    close(got[0] if Hk else got, turned64(q, pos, rope, 5e5, w), dtype)
    if Hk:
        close(got[1], turned64(k, pos, rope, 5e5), dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_far_positions(dtype):
    """Every position that fits 32 bits, backwards too. The frequencies are powers of two of a radian: fp64 angles are off by
    position * 2^-53 here, and the table's by the rounding of 1 / 2 pi, position * 2^-54 of a circle."""
    pos = [0, 1, -1, 2 ** 24 + 1, 10 ** 9 + 7, 2 ** 31 - 1, -2 ** 31, -12345]
    rope = moe.Rotary(16, frequencies=[2.0 ** -i for i in range(8)])
    q = tensor((len(pos), 2, 16), 1, dtype, DEV)
    want, bound = turned64(q, pos, rope, 0, frequencies=[2.0 ** -i for i in range(8)])
    far = np.abs(np.array(pos, dtype=np.float64))[:, None, None] * 2.0 ** -50
    close(rope.apply(q, i32(pos, DEV)), (want, bound + far * np.abs(f64(q)).sum(-1, keepdims=True)), dtype)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_turning_back_is_the_transpose(layout):
    """<turn(x), y> = <x, turn back(y)>, the gradient of a rotation."""
    rope = moe.Rotary(64, rotary_dim=48, layout=layout)
    x, y = tensor((50, 3, 64), 1, F32, DEV), tensor((50, 3, 64), 2, F32, DEV)
    p = i32(list(range(1000, 1050)), DEV)
    a, b = (rope.apply(x, p).double() * y.double()).sum(), (x.double() * rope.apply(y, -p).double()).sum()
    # each of the 9600 products is off by at most (64 + 32) h(fp32) of 2 |x y|
    assert abs(a - b) <= 2 * 96 * H32 * 2 * (x.abs().double().sum(-1) * y.abs().double().sum(-1)).sum()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_out_and_in_place(dtype, in_place):
    rope = moe.Rotary(128)
    T, H, Hk = 100, 8, 2
    x = tensor((T, H + 2 * Hk, 128), 5, dtype, DEV)
    v0 = x[:, H + Hk:].clone()
    q, k = x[:, :H], x[:, H:H + Hk]
    w = tensor((128,), 6, dtype, DEV)
    pos = i32(list(range(T)), DEV)
    want = rope.apply(q, pos, k, q_weight=w, k_weight=w)
    y = x if in_place else torch.full_like(x, float("nan"))
    got = rope.apply(q, pos, k, q_weight=w, k_weight=w, out=y[:, :H], k_out=y[:, H:H + Hk])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(x[:, H + Hk:], v0)
    if not in_place:
        assert torch.isnan(y[:, H + Hk:]).all()


def test_unturned_elements_are_kept_whatever_their_pairs_hold():
    rope = moe.Rotary(64, rotary_dim=16)
    q = tensor((4, 2, 64), 1, BF16, DEV)
    q[0, 0, 40] = float("inf")
    q[1, 1, 63] = float("nan")
    q[2, 0, 3] = float("inf")
    out = rope.apply(q, i32([5, 6, 7, 8], DEV))
    assert torch.equal(out[..., 16:].nan_to_num(7.0), q[..., 16:].nan_to_num(7.0))
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[0, 0, 40] = want[1, 1, 63] = want[2, 0, 3] = want[2, 0, 11] = True
    assert torch.equal(bad, want)


def test_nothing_to_do():
    rope = moe.Rotary(64)
    e = torch.empty((0, 4, 64), dtype=BF16, device=DEV)
    out, k = rope.apply(e, i32([], DEV), e)
    assert out.shape == e.shape and k.shape == e.shape


# ---------------------------------------------------------------------------------------------- append

def filled(lens, page, Hk, D, dtype, seed, layers=1, spare=3):
    r = random.Random(seed)
    m = Model(layers, sum(-(-n // page) for n in lens) + spare, page, len(lens), max(1, max(-(-n // page) for n in lens)) + 1)
    free = list(range(len(m.refs)))
    r.shuffle(free)
    for s, n in enumerate(lens):
        m.rows[s] = [free.pop() for _ in range(-(-n // page))]
        m.lens[s] = n
        for p in m.rows[s]:
            m.refs[p] = 1
    shape = (layers, len(m.refs), Hk, page, D)
    m.k, m.v = tensor(shape, seed, dtype, "cpu"), tensor(shape, seed + 1, dtype, "cpu")
    cache = moe.KVCache(m.k.to(DEV), m.v.to(DEV), i32(m.table(), DEV), i32(m.lens, DEV), i32(m.refs, DEV))
    return m, cache


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("D,R,page,H,Hk", [(64, 64, 16, 4, 2), (128, 128, 64, 8, 2), (80, 20, 32, 3, 3), (96, 96, 128, 0, 1),
                                           (256, 64, 16, 2, 1), (40, 6, 256, 5, 5), (72, 0, 16, 6, 2)])
def test_append(D, R, page, H, Hk, norm, layout, dtype):
    r = random.Random(D + page)
    held = [0, 3, page - 1, page, 2 * page + 5, 9]
    new = [1, page + 3, 2, 0, 5, 1]
    m, cache = filled([a + b for a, b in zip(held, new)], page, Hk, D, dtype, D, layers=2)
    order = list(range(6))
    r.shuffle(order)
    new, held = [new[s] for s in order], [held[s] for s in order]
    offs, T = offsets(new), sum(new)
    x = tensor((T, H + 2 * Hk, D), 3, dtype, DEV)
    q, k, v = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
    wq, wk = (tensor((D,), s, dtype, DEV) if norm else None for s in (1, 2))
    rope = moe.Rotary(D, rotary_dim=R, layout=layout)
    out = cache.append(k, v, i32(order, DEV), i32(offs, DEV), i32(held, DEV), rope, layer=1, q=q if H else None,
                       q_weight=wq if H else None, k_weight=wk)
    assert cache.device_status() == (moe.MOE_OK, 0)
    pos = [p + t for p, n in zip(held, new) for t in range(n)]
    kn, bound = turned64(k, pos, rope, 1e4, wk)
    if H:
        close(out, turned64(q, pos, rope, 1e4, wq), dtype)
    else:
        assert out is None
    # pages: v exactly, k within its bounds, and nothing else changed
    got_k, got_v = cache.k.cpu(), cache.v.cpu()
    at = [(m.rows[s][p // page], p % page) for s, p0, n in zip(order, held, new) for p in range(p0, p0 + n)]
    pages, rows = [a for a, _ in at], [b for _, b in at]
    close(got_k[1, pages, :, rows], (kn, bound), dtype)
    assert torch.equal(got_v[1, pages, :, rows], v.cpu())
    got_k[1, pages, :, rows] = m.k[1, pages, :, rows]
    got_v[1, pages, :, rows] = m.v[1, pages, :, rows]
    assert torch.equal(got_k, m.k) and torch.equal(got_v, m.v)
    assert cache.lens.tolist() == m.lens and cache.table.tolist() == m.table() and cache.refs.tolist() == m.refs


def test_append_without_rotary_is_write():
    m, a = filled([70, 5], 16, 2, 64, BF16, 1)
    b = moe.KVCache(a.k.clone(), a.v.clone(), a.table, a.lens, a.refs)
    x = tensor((11, 4, 64), 2, BF16, DEV)
    args = (x[:, :2], x[:, 2:], i32([1, 0], DEV), i32([0, 5, 11], DEV), i32([0, 64], DEV))
    a.write(*args)
    b.append(*args)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)


def test_append_skips_what_write_skips():
    """Positions past a slot's length, a shared page, a bad slot, a bad page: that token's rows stay, and q_out's too."""
    page, D = 16, 64
    for spoil, bad in (("length", [3, 4]), ("shared", [0, 1, 2]), ("slot", [5, 6]), ("page", [3, 4])):
        m, cache = filled([16, 20, 40], page, 1, D, BF16, 3)
        slots, offs, pos = [0, 1, 2], [0, 3, 5, 7], [13, 18, 38]
        if spoil == "length":
            cache.lens[1] = 18
        elif spoil == "shared":
            cache.refs[m.rows[0][0]] = 2
        elif spoil == "slot":
            slots[2] = 3
        else:
            cache.table[1, 1] = 10 ** 6
        k0, v0 = cache.k.clone(), cache.v.clone()
        x = tensor((7, 4, D), 4, BF16, DEV)
        rope = moe.Rotary(D)
        qo = torch.full((7, 2, D), 7.0, dtype=BF16, device=DEV)
        cache.append(x[:, 2:3], x[:, 3:], i32(slots, DEV), i32(offs, DEV), i32(pos, DEV), rope, q=x[:, :2], q_out=qo)
        status, detail = cache.device_status()
        assert status == moe.MOE_ERR_DEVICE_CHECK and detail in bad
        want, _ = turned64(x[:, :2], [13, 14, 15, 18, 19, 38, 39], rope, 1e4)
        for t in range(7):
            if t in bad:
                assert (qo[t] == 7).all()
            else:
                assert np.abs(f64(qo[t]) - want[t]).max() < 0.05
        changed = (cache.k != k0).any(-1).sum() + (cache.v != v0).any(-1).sum()
        assert changed == 2 * (7 - len(bad))
