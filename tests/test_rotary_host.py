"""Rotary tables, and the refusals of Rotary, KVCache.append and Attention.chunk, which need no GPU."""
import copy
import ctypes
import math
import pickle

import pytest
import torch

import sparse_mixture_experts_moe_gb300 as moe
from sparse_mixture_experts_moe_gb300 import _lib
from sparse_mixture_experts_moe_gb300.rotary import _Rotary
from test_attention_device_host import Fake, cache_on, calls  # noqa: F401
from test_attention_host import BAD, BAD_CACHES, FAKE, OK, cache


def wanted(R, base, scaling, factor, L, low, high):
    if scaling == "base":
        base *= factor ** (R / (R - 2))
    out = []
    first = max(0, math.floor(R * math.log(L / (math.tau * high)) / (2 * math.log(base)))) if scaling == "pairs" else 0
    last = min(R - 1, math.ceil(R * math.log(L / (math.tau * low)) / (2 * math.log(base)))) if scaling == "pairs" else 0
    for p in range(R // 2):
        f = base ** (-2 * p / R)
        if scaling == "linear":
            f /= factor
        elif scaling == "turns":
            s = min(1.0, max(0.0, (L * f / math.tau - low) / (high - low)))
            f *= s + (1 - s) / factor
        elif scaling == "pairs":
            r = 0.0 if p <= first else 1.0 if p >= last else (p - first) / (last - first)
            f *= 1 - r + r / factor
        out.append(f)
    return out


@pytest.mark.parametrize("R", [2, 4, 20, 64, 128, 256])
@pytest.mark.parametrize("scaling,low,high", [(None, 1, 4), ("linear", 1, 4), ("base", 1, 4), ("turns", 1, 4), ("turns", 2, 9),
                                              ("pairs", 1, 32), ("pairs", 0.5, 3)])
@pytest.mark.parametrize("base,factor,L", [(1e4, 8.0, 4096), (5e5, 32.0, 8192), (1e4, 1.0, 64)])
def test_frequencies(R, scaling, low, high, base, factor, L):
    if scaling == "base" and R == 2:
        with pytest.raises(ValueError):
            moe.Rotary(256, rotary_dim=R, base=base, scaling=scaling, factor=factor)
        return
    r = moe.Rotary(256, rotary_dim=R, base=base, scaling=scaling, factor=factor, original_len=L, low=low, high=high)
    want = wanted(R, base, scaling, factor, L, low, high)
    # double's roundings in the power, the division by 2 pi and back: a few 2^-53 each, and the table's 2^-64 of a circle
    assert all(abs(a - b) <= 16 * 2.0 ** -53 * b + math.tau * 2.0 ** -64 for a, b in zip(r.frequencies, want))
    assert r.magnitude == pytest.approx(0.1 * math.log(factor) + 1 if scaling == "pairs" else 1.0, rel=2.0 ** -23)
    # the ends: nothing changes for factor 1; the fastest pair is kept, the slowest divided, where the turns say so
    if factor == 1.0:
        assert r.frequencies == moe.Rotary(256, rotary_dim=R, base=base).frequencies
    if scaling == "base":
        assert r.frequencies[-1] == pytest.approx(base ** (-2 * (R // 2 - 1) / R) / factor, rel=1e-12)


def test_own_frequencies_and_whole_turns():
    f = [0.5, 7.0, -0.25, 0.0]
    r = moe.Rotary(8, frequencies=f, magnitude=0.5)
    assert r.magnitude == 0.5
    assert r.frequencies == pytest.approx([x % math.tau for x in f], rel=1e-14)
    tiny = moe.Rotary(8, rotary_dim=2, frequencies=[-1e-300])
    assert tiny.frequencies == [0.0]


@pytest.mark.parametrize("again", [copy.copy, copy.deepcopy, lambda r: pickle.loads(pickle.dumps(r))])
def test_copies_have_tables_of_their_own(again):
    for r in (moe.Rotary(64, rotary_dim=32, scaling="pairs", factor=4, original_len=2048), moe.Rotary(8, frequencies=iter([1, 2, 3, 4.5]))):
        c = again(r)
        assert c._ref == ctypes.addressof(c._c) != r._ref
        assert c.frequencies == r.frequencies and c.magnitude == r.magnitude and c.layout == r.layout


@pytest.mark.parametrize("kw", [
    dict(head_dim=12), dict(head_dim=4), dict(head_dim=264), dict(rotary_dim=-2), dict(rotary_dim=66), dict(rotary_dim=7),
    dict(layout="whole"), dict(scaling="ntk"), dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")),
    dict(magnitude=0.0), dict(magnitude=float("inf")), dict(magnitude=float("nan")), dict(scaling="linear", factor=0.5),
    dict(scaling="linear", factor=float("inf")), dict(scaling="turns", factor=2.0), dict(scaling="pairs", factor=2.0),
    dict(scaling="turns", factor=2.0, original_len=100, low=4, high=4), dict(scaling="pairs", factor=2.0, original_len=100, low=0),
    dict(frequencies=[1.0]), dict(frequencies=[float("nan")] * 32), dict(frequencies=[1.0] * 32, scaling="linear")])
def test_rotary_refusals(kw):
    with pytest.raises(ValueError):
        moe.Rotary(**{**dict(head_dim=64), **kw})


def table(**kw):
    r = _Rotary()
    assert _lib.lib().moe_rotary_init(ctypes.addressof(r), 64, 64, 0, 1e4, 0, 1.0, 0, 1.0, 4.0, 0.0) == OK
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def apply(r, **kw):
    a = dict(q=FAKE, qs=512, H=8, k=FAKE, ks=128, Hk=2, pos=FAKE, T=5, dt=1, wq=None, wk=None, eps=1e-6, qo=FAKE, qos=512,
             ko=FAKE, kos=128)
    a.update(kw)
    return _lib.lib().moe_rotary_apply(None if r is None else ctypes.addressof(r), *a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q=FAKE + 2), dict(qs=511), dict(qs=504), dict(H=0), dict(H=70000), dict(k=None), dict(k=FAKE + 4), dict(ks=120),
    dict(Hk=-1), dict(Hk=0), dict(Hk=70000), dict(pos=None), dict(T=-1), dict(dt=2), dict(dt=-1), dict(wq=FAKE + 2), dict(wk=FAKE + 8),
    dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")), dict(qo=None), dict(qo=FAKE + 8), dict(qos=500), dict(ko=None),
    dict(ko=FAKE + 2), dict(kos=100), dict(qs=1 << 41)])
def test_apply_refusals(kw):
    assert apply(table(), **kw) == BAD


def test_apply_refuses_broken_tables():
    assert apply(None) == BAD
    for kw in (dict(D=12), dict(D=0), dict(R=66), dict(R=3), dict(R=-2), dict(layout=2), dict(magnitude=float("nan"))):
        assert apply(table(**kw)) == BAD
    assert apply(table(), T=0) == OK
    assert apply(table(), T=0, k=None, ko=None, Hk=0, q=None, pos=None) == OK


def append(c, r, **kw):
    usual = cache()
    n = _lib.lib().moe_cache_workspace_bytes(ctypes.addressof(usual))
    a = dict(layer=0, slots=FAKE, offsets=FAKE, pos=FAKE, n=2, total=5, r=None if r is None else ctypes.addressof(r), k=FAKE, v=FAKE,
             ks=128, vs=128, wk=None, q=FAKE, qs=512, H=8, wq=None, eps=1e-6, qo=FAKE, qos=512, ws=FAKE, bytes=n)
    a.update(kw)
    return _lib.lib().moe_cache_append(ctypes.addressof(c), *a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(layer=2), dict(layer=-1), dict(slots=None), dict(offsets=None), dict(pos=None), dict(n=9), dict(n=-1), dict(n=0),
    dict(total=-1), dict(k=None), dict(v=None), dict(ks=127), dict(vs=132), dict(k=FAKE + 8), dict(wk=FAKE + 2), dict(q=None),
    dict(q=FAKE + 2), dict(qs=500), dict(H=-1), dict(H=0), dict(H=70000), dict(wq=FAKE + 4), dict(eps=-1.0), dict(eps=float("nan")),
    dict(qo=None), dict(qo=FAKE + 2), dict(qos=511), dict(ws=None), dict(bytes=1000)])
def test_append_refusals(kw):
    assert append(cache(), table(), **kw) == BAD


def test_append_tables_and_nothing_to_do():
    assert append(cache(), table(D=32, R=32)) == BAD   # another head's table
    assert append(cache(), table(R=66)) == BAD
    assert append(cache(), table(), total=0, n=0) == OK
    assert append(cache(), None, total=0, n=0, q=None, qo=None, H=0) == OK


def chunk(c, **kw):
    usual = cache()
    a = dict(layer=0, q=FAKE, slots=FAKE, qo=FAKE, n=3, Tq=7, H=8, qs=512, os=512, scale=0.125, flags=1, out=FAKE, lse=None, ws=FAKE,
             bytes=_lib.lib().moe_attention_chunk_workspace_bytes(ctypes.addressof(usual), 3, 7, 8))
    a.update(kw)
    return _lib.lib().moe_attention_chunk(ctypes.addressof(c), *a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(layer=-1), dict(layer=2), dict(q=None), dict(slots=None), dict(qo=None), dict(out=None), dict(n=-1), dict(n=0), dict(Tq=-1),
    dict(H=7), dict(H=0), dict(H=70000), dict(qs=511), dict(os=500), dict(scale=0.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(flags=2), dict(flags=-1), dict(ws=None), dict(bytes=1000), dict(q=FAKE + 2), dict(out=FAKE + 4),
    dict(ws=FAKE + 4), dict(Tq=1 << 30)])
def test_chunk_refusals(kw):
    assert chunk(cache(), **kw) == BAD


def test_chunk_sizes():
    lib, c = _lib.lib(), cache()
    size = lib.moe_attention_chunk_workspace_bytes
    ref = ctypes.addressof(c)
    assert chunk(c, n=0, Tq=0) == OK and chunk(c, n=3, Tq=0) == OK
    assert size(ref, 0, 0, 8) >= 256 and size(ref, 3, 7, 8) % 256 == 0
    for args in ((-1, 7, 8), (3, -1, 8), (3, 7, 7), (3, 7, 0), (3, 1 << 30, 8)):
        assert size(ref, *args) == 0
    # pieces of at most 256 rows, however long the chunk
    assert size(ref, 3, 1 << 20, 8) == size(ref, 3, 64, 8)
    for kw in BAD_CACHES:
        b = cache(**kw)
        assert chunk(b, Tq=0) == BAD
        assert append(b, table(), total=0, n=0) == BAD
        if not set(kw) & {"k", "v", "table", "lens", "refs"}:
            assert size(ctypes.addressof(b), 3, 7, 8) == 0


# ---------------------------------------------------------------------------------------------- the binding

F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32


def rotary(called, many=False, current=0, **kw):
    r = moe.Rotary(64, **kw)
    r._raw_stream = lambda dev: 0
    r._current_device, r._many = (lambda: current), many
    r._call = lambda *a: called.append(a) or moe.MOE_OK
    r._new = lambda shape, strides, dtype: Fake(shape, dtype, 0)
    return r


def test_binding_apply_refusals():
    called = []
    r = rotary(called)
    q, k, p, w = Fake((3, 4, 64), BF16, 0), Fake((3, 2, 64), BF16, 0), Fake((3,), I32, 0), Fake((64,), BF16, 0)
    r.apply(q, p, k, q_weight=w)
    assert len(called) == 1
    for bad in [lambda: r.apply(Fake((3, 4, 32), BF16, 0), p), lambda: r.apply(Fake((3, 256), BF16, 0), p),
                lambda: r.apply(q, Fake((4,), I32, 0)), lambda: r.apply(q, Fake((3,), torch.int64, 0)), lambda: r.apply(q, Fake((3, 1), I32, 0)),
                lambda: r.apply(q, Fake((3,), I32, 1)), lambda: r.apply(q, p, Fake((2, 2, 64), BF16, 0)), lambda: r.apply(q, p, Fake((3, 2, 64), F32, 0)),
                lambda: r.apply(q, p, Fake((3, 0, 64), BF16, 0)), lambda: r.apply(Fake((3, 0, 64), BF16, 0), p),
                lambda: r.apply(q, p, k, q_weight=Fake((64,), F32, 0)), lambda: r.apply(q, p, k, k_weight=Fake((32,), BF16, 0)),
                lambda: r.apply(q, p, k_weight=w), lambda: r.apply(q, p, k_out=k), lambda: r.apply(q, p, stream=5), lambda: r.apply(q, p, k, out=q, stream=5),
                lambda: r.apply(torch.zeros(3, 4, 64), torch.zeros(3, dtype=I32))]:
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        r.apply(Fake((3, 4, 64), torch.float16, 0), p)
    assert len(called) == 1
    assert r.apply(q, p) is not None and len(called) == 2   # a call that was refused leaves nothing behind


@pytest.mark.parametrize("dev", [0, 1])
def test_binding_devices(calls, dev):  # noqa: F811
    called, watch = calls
    r = rotary(called, many=True)
    a, c = watch(moe.Attention(4, 2, 64, F32)), cache_on(dev, watch)
    a._chunk = c._append = lambda *x: called.append(x) or moe.MOE_OK
    kv, i = Fake((3, 2, 64), F32, dev), lambda n: Fake((n,), I32, dev)
    q = Part(3, 0, 4, 4, at=1 << 18, dev=dev)
    kv.element_size = lambda: 4
    for call in [lambda: r.apply(q, i(3), out=q), lambda: c.append(kv, kv, i(2), i(3), i(2), q=q, q_out=q), lambda: c.append(kv, kv, i(2), i(3), i(2)),
                 lambda: a.chunk(q, c, i(2), i(3), out=q), lambda: a.chunk(q, c, i(2), i(3), out=q, stream=5)]:
        if dev == 0:
            call()
        else:
            with pytest.raises(ValueError, match="current device"):
                call()
    assert len(called) == (5 if dev == 0 else 0)


def test_binding_append_and_chunk_refusals(calls):  # noqa: F811
    called, watch = calls
    a, c = watch(moe.Attention(4, 2, 64, F32)), cache_on(0, watch)
    a._chunk = c._append = lambda *x: called.append(x) or moe.MOE_OK
    q, kv, i = Fake((3, 4, 64), F32, 0), Fake((3, 2, 64), F32, 0), lambda n: Fake((n,), I32, 0)
    rope, other = moe.Rotary(64), moe.Rotary(32)
    args = (kv, kv, i(2), i(3), i(2))
    for bad in [lambda: c.append(kv, Fake((2, 2, 64), F32, 0), *args[2:]), lambda: c.append(kv, kv, i(2), i(2), i(2)),
                lambda: c.append(kv, kv, i(2), i(3), i(3)), lambda: c.append(*args, other), lambda: c.append(*args, "rope"),
                lambda: c.append(*args, rope, q=Fake((2, 4, 64), F32, 0)), lambda: c.append(*args, rope, q=Fake((3, 4, 64), BF16, 0)),
                lambda: c.append(*args, rope, q_out=q), lambda: c.append(*args, rope, q_weight=Fake((64,), F32, 0)),
                lambda: c.append(*args, rope, q=q, q_weight=Fake((64,), BF16, 0)), lambda: c.append(*args, rope, k_weight=Fake((32,), F32, 0)),
                lambda: c.append(*args, rope, q=q, stream=3), lambda: c.append(*args, rope, q=q, q_out=Fake((3, 2, 64), F32, 0)),
                lambda: a.chunk(Fake((3, 2, 64), F32, 0), c, i(2), i(3)), lambda: a.chunk(q, c, i(2), i(2)),
                lambda: a.chunk(q, c, i(2), Fake((3,), torch.int64, 0)), lambda: a.chunk(q, c, Fake((2,), I32, 1), i(3)),
                lambda: a.chunk(q, c, i(2), i(3), stream=4), lambda: a.chunk(q, c, i(2), i(3), out=Fake((2, 4, 64), F32, 0)),
                lambda: moe.Attention(4, 2, 32, F32).chunk(q, c, i(2), i(3))]:
        with pytest.raises(ValueError):
            bad()
    assert not called


class Part(Fake):
    """A slice of heads of a fused tensor [T, row, 64] of float32 at address `at`."""

    def __init__(self, T, first, n, row, at=0, dev=0):
        super().__init__((T, n, 64), F32, dev)
        self.at, self.row = (1 << 20) + at + first * 256, row

    def stride(self):
        return self.row * 64, 64, 1

    def element_size(self):
        return 4

    def data_ptr(self):
        return self.at


@pytest.mark.parametrize("T", [1, 2, 9])
def test_outputs_may_be_inputs_but_not_overlap_them(T):
    called = []
    r = rotary(called)
    p = Fake((T,), I32, 0)
    q, k = Part(T, 0, 4, 8), Part(T, 4, 2, 8)
    far = 1 << 18
    for out, k_out in [(q, k), (Part(T, 0, 4, 8, far), Part(T, 4, 2, 8, far)), (q, Part(T, 6, 2, 8)), (Part(T, 0, 4, 4, far), k)]:
        r.apply(q, p, k, out=out, k_out=k_out)
    assert len(called) == 4
    for out, k_out in [(Part(T, 1, 4, 8), k), (q, Part(T, 3, 2, 8)), (q, Part(T, 5, 2, 8)), (Part(T, 0, 4, 8, far), Part(T, 2, 2, 8, far)),
                       (Part(T, 0, 4, 8, 256), Part(T, 0, 2, 8, far))]:
        with pytest.raises(ValueError):
            r.apply(q, p, k, out=out, k_out=k_out)
    if T > 1:
        with pytest.raises(ValueError):
            r.apply(q, p, k, out=Part(T, 0, 4, 9), k_out=Part(T, 0, 2, 8, far))
    assert len(called) == 4
