"""Refusals of the attention and cache calls, which need no GPU: every bad argument is turned down on the host."""
import ctypes

import pytest
import torch

import sparse_mixture_experts_moe_gb300 as moe
from sparse_mixture_experts_moe_gb300 import _lib
from sparse_mixture_experts_moe_gb300.attention import _Cache

FAKE = 1 << 20  # non-null, aligned, never dereferenced
BAD, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_OK


def prompt(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qo=FAKE, ko=None, n=2, Tq=10, Tkv=10, H=8, Hk=2, D=64, qs=512, ks=128, vs=128,
             os=512, scale=0.125, flags=1, dt=1, out=FAKE, lse=None, ws=FAKE, bytes=256)
    a.update(kw)
    return _lib.lib().moe_attention_prompt(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(k=None), dict(v=None), dict(qo=None), dict(out=None), dict(ws=None), dict(bytes=255), dict(n=-1),
    dict(n=0), dict(Tq=-1), dict(Tkv=-1), dict(Tkv=11), dict(H=7), dict(H=0), dict(Hk=0), dict(Hk=3), dict(D=0),
    dict(D=12), dict(D=264), dict(qs=511), dict(qs=504), dict(ks=120), dict(vs=130), dict(os=508), dict(scale=0.0),
    dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(flags=2), dict(flags=-1), dict(dt=2),
    dict(q=FAKE + 2), dict(k=FAKE + 8), dict(v=FAKE + 4), dict(out=FAKE + 2), dict(ws=FAKE + 8), dict(H=70000),
    dict(qs=1 << 41), dict(Tq=1 << 29, Tkv=1 << 29)])
def test_prompt_refusals(kw):
    assert prompt(**kw) == BAD


def test_prompt_no_tokens_is_a_no_op():
    assert prompt(Tq=0, Tkv=0, n=0) == OK
    assert prompt(Tq=0, Tkv=0, n=3) == OK
    assert prompt(Tq=0, Tkv=5, n=3, ko=FAKE) == OK


def cache(**kw):
    a = dict(k=FAKE, v=FAKE, table=FAKE, lens=FAKE, refs=FAKE, n_layers=2, n_pages=100, page_size=16, n_slots=8,
             table_width=12, H_kv=2, D=64, dt=1)
    a.update(kw)
    return _Cache(*a.values())


BAD_CACHES = [dict(k=None), dict(v=None), dict(table=None), dict(lens=None), dict(refs=None), dict(k=FAKE + 8),
              dict(n_layers=0), dict(n_pages=0), dict(n_pages=1 << 30), dict(page_size=8), dict(page_size=24),
              dict(page_size=512), dict(n_slots=0), dict(table_width=0), dict(H_kv=0), dict(D=4), dict(D=12),
              dict(D=264), dict(dt=3), dict(n_slots=1 << 20, table_width=1 << 12), dict(table_width=1 << 28),
              dict(n_pages=1 << 29)]


def decode(c, **kw):
    n = kw.get("n", 3)
    a = dict(layer=0, q=FAKE, slots=FAKE, n=n, H=8, qs=512, os=512, shared=32, scale=0.125, out=FAKE, lse=None, ws=FAKE,
             bytes=_lib.lib().moe_attention_workspace_bytes(3, 8, 64))
    a.update(kw)
    return _lib.lib().moe_attention_decode(ctypes.addressof(c), *a.values(), None)


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_bad_caches(kw):
    c, lib = cache(**kw), _lib.lib()
    ref, big = ctypes.addressof(c), 1 << 40
    assert decode(c, n=0) == BAD
    assert lib.moe_cache_clear(ref, None) == BAD
    assert lib.moe_cache_resize(ref, FAKE, FAKE, 0, FAKE, big, None) == BAD
    assert lib.moe_cache_fork(ref, FAKE, FAKE, 0, FAKE, big, None) == BAD
    assert lib.moe_cache_compact(ref, FAKE, FAKE, big, None) == BAD
    assert lib.moe_cache_copy_pages(ref, FAKE, FAKE, 0, FAKE, big, None) == BAD
    assert lib.moe_cache_write(ref, 0, FAKE, FAKE, FAKE, 0, 0, FAKE, FAKE, 128, 128, FAKE, big, None) == BAD
    if not set(kw) & {"k", "v", "table", "lens", "refs"}:
        assert lib.moe_cache_workspace_bytes(ref) == 0
        assert lib.moe_cache_workspace_init(ref, FAKE, big, None) == BAD


@pytest.mark.parametrize("kw", [
    dict(layer=-1), dict(layer=2), dict(q=None), dict(slots=None), dict(out=None), dict(n=-1), dict(H=7), dict(H=0),
    dict(qs=511), dict(os=500), dict(shared=-16), dict(shared=8), dict(shared=13 * 16), dict(scale=0.0),
    dict(scale=float("nan")), dict(ws=None), dict(bytes=1000), dict(q=FAKE + 2), dict(out=FAKE + 4), dict(ws=FAKE + 4)])
def test_decode_refusals(kw):
    assert decode(cache(), **kw) == BAD


def test_cache_call_refusals():
    c, lib = cache(), _lib.lib()
    ref, n = ctypes.addressof(c), _lib.lib().moe_cache_workspace_bytes(ctypes.addressof(c))
    assert n > 0 and n % 256 == 0
    for args in [(FAKE, FAKE, 9, FAKE, n), (FAKE, FAKE, -1, FAKE, n), (None, FAKE, 1, FAKE, n), (FAKE, None, 1, FAKE, n),
                 (FAKE, FAKE, 1, None, n), (FAKE, FAKE, 1, FAKE, n - 1), (FAKE, FAKE, 1, FAKE + 8, n)]:
        assert lib.moe_cache_resize(ref, *args, None) == BAD
        assert lib.moe_cache_fork(ref, *args, None) == BAD
        assert lib.moe_cache_copy_pages(ref, args[0], args[1], args[2] if args[2] != 9 else 101, *args[3:], None) == BAD
    assert lib.moe_cache_compact(ref, FAKE, FAKE, n - 1, None) == BAD
    ok = dict(layer=0, slots=FAKE, offsets=FAKE, pos=FAKE, n=2, total=5, k=FAKE, v=FAKE, ks=128, vs=128, ws=FAKE, bytes=n)
    for kw in [dict(layer=2), dict(layer=-1), dict(slots=None), dict(offsets=None), dict(pos=None), dict(n=9), dict(n=-1),
               dict(n=0), dict(total=-1), dict(k=None), dict(v=None), dict(ks=127), dict(vs=132), dict(k=FAKE + 8),
               dict(ws=None), dict(bytes=n - 1)]:
        assert lib.moe_cache_write(ref, *{**ok, **kw}.values(), None) == BAD, kw
    # nothing to do is not an error
    assert lib.moe_cache_resize(ref, None, None, 0, FAKE, n, None) == OK
    assert lib.moe_cache_fork(ref, None, None, 0, FAKE, n, None) == OK
    assert lib.moe_cache_copy_pages(ref, None, None, 0, FAKE, n, None) == OK
    assert lib.moe_cache_write(ref, *{**ok, "total": 0, "n": 0}.values(), None) == OK
    assert decode(c, n=0) == OK


def test_plans():
    lib, n = _lib.lib(), _lib.lib().moe_cache_plan_bytes()
    buf = ctypes.create_string_buffer(n)
    at = ctypes.addressof(buf)
    c = cache(dt=0)  # an fp32 cache needs no descriptors, so its plan can be made without a GPU
    assert lib.moe_cache_plan(ctypes.addressof(c), at, n) == OK
    for args in [(None, at, n), (ctypes.addressof(c), None, n), (ctypes.addressof(c), at, n - 1)]:
        assert lib.moe_cache_plan(*args) == BAD
    bad = cache(page_size=24)
    assert lib.moe_cache_plan(ctypes.addressof(bad), at, n) == BAD
    # a plan of another cache is refused
    for kw in [dict(k=FAKE + 256), dict(n_pages=101), dict(n_layers=1), dict(page_size=32), dict(H_kv=4), dict(D=32)]:
        other = cache(**kw)
        other.plan = at
        assert decode(other, H=8, qs=512, os=512, shared=0) == BAD


def test_null_cache():
    lib = _lib.lib()
    assert lib.moe_cache_workspace_bytes(None) == 0
    assert lib.moe_cache_clear(None, None) == BAD
    assert lib.moe_attention_workspace_bytes(4, 0, 64) == 0
    assert lib.moe_attention_workspace_bytes(-1, 8, 64) == 0
    assert lib.moe_attention_workspace_bytes(0, 8, 64) > 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    a = moe.Attention(8, 2, 64, torch.bfloat16)
    x = torch.zeros((4, 8, 64), dtype=torch.bfloat16)
    kv = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    o = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        a.prompt(x, kv, kv, o)
    with pytest.raises(ValueError):
        moe.Attention(7, 2, 64, torch.bfloat16)
    with pytest.raises(ValueError):
        moe.Attention(8, 2, 60, torch.bfloat16)
    with pytest.raises(TypeError):
        moe.Attention(8, 2, 64, torch.float16)
    with pytest.raises(ValueError):
        i = torch.zeros(3, dtype=torch.int32)
        p = torch.zeros((1, 4, 2, 16, 64), dtype=torch.bfloat16)
        moe.KVCache(p, p, torch.zeros((3, 2), dtype=torch.int32), i, i)  # refs must have one count a page


def test_no_stream_records_without_a_gpu():
    assert _lib.lib().moe_stream_capture_id(None) == 0


def test_prompt_workspace_bytes():
    f = _lib.lib().moe_attention_prompt_workspace_bytes
    assert f(0, 0, 0, 8, 2, 64, moe.MOE_DTYPE_BF16) == 256
    assert f(1, 16, 1000, 8, 2, 64, moe.MOE_DTYPE_BF16) == 256      # few keys
    assert f(1, 16, 100000, 8, 2, 64, moe.MOE_DTYPE_F32) == 256     # fp32 needs none
    assert f(1, 16, 100000, 8, 2, 136, moe.MOE_DTYPE_BF16) == 256
    assert f(1, 16, 100000, 8, 2, 64, moe.MOE_DTYPE_BF16) % 256 == 0
    for args in [(-1, 16, 16, 8, 2, 64, 0), (1, -1, 16, 8, 2, 64, 0), (1, 16, -1, 8, 2, 64, 0), (1, 16, 16, 7, 2, 64, 0),
                 (1, 16, 16, 8, 2, 60, 0), (1, 16, 16, 8, 2, 264, 0), (1, 16, 16, 8, 2, 64, 7), (1, 1 << 30, 16, 8, 2, 64, 0),
                 (1, 16, 16, 8, 0, 64, 0)]:
        assert f(*args) == 0, args
