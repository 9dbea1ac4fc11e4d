"""Calls on tensors of a device that is not the current one, whose kernels would run on another device than the memory
they are given. Needs no GPU: tensors are stand-ins, and the library's calls are counted, not made."""
import threading
import time

import pytest
import torch

import sparse_mixture_experts_moe_gb300 as moe


class Fake:
    """What the binding looks at of a dense tensor on cuda:`dev`."""
    is_cuda = True

    def __init__(self, shape, dtype, dev):
        self.shape, self.dtype, self.device, self._dev = torch.Size(shape), dtype, torch.device("cuda", dev), dev

    def get_device(self):
        return self._dev

    def dim(self):
        return len(self.shape)

    def stride(self):
        s = [1]
        for n in reversed(self.shape[1:]):
            s.insert(0, s[0] * n)
        return tuple(s)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


@pytest.fixture
def calls(monkeypatch):
    """Names of the library's kernels that were called; the current device is 0."""
    called = []

    class Space:
        def get(self, stream, nbytes, dev, *more):
            return None, 1 << 40, 1 << 21

    def watch(obj):
        obj._raw_stream = lambda dev: 0
        obj._current_device, obj._many = (lambda: 0), True
        obj._capturing, obj._recording = (lambda: False), (lambda handle: 0)
        obj._ws, obj._of = Space(), {}

        class Lib:
            def __getattr__(self, name):
                return (lambda *a: 256) if name.endswith("_bytes") else (lambda *a: 0) if name.endswith("_id") else (lambda *a: called.append(name) or moe.MOE_OK)
        obj._lib = Lib()
        for name in ("_prompt", "_decode"):
            if hasattr(obj, name):
                setattr(obj, name, lambda *a, name=name: called.append(name) or moe.MOE_OK)
        return obj
    return called, watch


def cache_on(dev, watch):
    i = torch.int32
    kv = Fake((1, 4, 2, 16, 64), torch.float32, dev)
    return watch(moe.KVCache(kv, kv, Fake((3, 2), i, dev), Fake((3,), i, dev), Fake((4,), i, dev)))


@pytest.mark.parametrize("dev", [0, 1])
def test_attention_calls(calls, dev):
    called, watch = calls
    a = watch(moe.Attention(4, 2, 64, torch.float32))
    c = cache_on(dev, watch)
    q, kv, i = Fake((3, 4, 64), torch.float32, dev), Fake((3, 2, 64), torch.float32, dev), lambda n: Fake((n,), torch.int32, dev)
    todo = [lambda: a.prompt(q, kv, kv, i(2), out=q), lambda: a.prompt(q, kv, kv, i(2), out=q, stream=5),
            lambda: a.decode(q, c, i(3), out=q), lambda: a.decode(q, c, i(3), out=q, stream=5)]
    for call in todo:
        if dev == 0:
            call()
        else:
            with pytest.raises(ValueError, match="current device"):
                call()
    assert called == (["_prompt", "_prompt", "_decode", "_decode"] if dev == 0 else [])


@pytest.mark.parametrize("dev", [0, 1])
def test_cache_calls(calls, dev):
    called, watch = calls
    c = cache_on(dev, watch)
    kv, i = Fake((3, 2, 64), torch.float32, dev), lambda n: Fake((n,), torch.int32, dev)
    todo = [c.clear, lambda: c.resize(i(2), i(2)), lambda: c.write(kv, kv, i(2), i(3), i(2)), lambda: c.fork(i(2), i(2)),
            lambda: c.compact(i(1)), lambda: c.copy_pages(i(2), i(2)), lambda: c.resize(i(2), i(2), stream=5)]
    for call in todo:
        if dev == 0:
            call()
        else:
            with pytest.raises(ValueError, match="current device"):
                call()
    assert len(called) == (len(todo) if dev == 0 else 0)


@pytest.mark.parametrize("stream", [None, 9])
def test_calls_say_whether_they_are_recorded(calls, stream):
    called, watch = calls
    a = watch(moe.Attention(4, 2, 64, torch.float32))
    c = cache_on(0, watch)
    asked = []
    a._ws.get = lambda *args: asked.append(args[3]) or (None, 1 << 40, 1 << 21)
    q, kv, i = Fake((3, 4, 64), torch.float32, 0), Fake((3, 2, 64), torch.float32, 0), lambda n: Fake((n,), torch.int32, 0)
    for now in (0, 41):
        a._capturing, a._recording = (lambda: now != 0), (lambda handle: now)
        a.prompt(q, kv, kv, i(2), out=q, stream=stream)
        a.decode(q, c, i(3), out=q, stream=stream)
    assert asked == [0, 0, 41, 41]


def test_threads_that_use_one_object_take_turns(calls):
    """A call enqueues several kernels, and the library's calls run without the interpreter's lock: the kernels of two calls
    must not mix, as they use one workspace."""
    called, watch = calls
    a = watch(moe.Attention(4, 2, 64, torch.float32))
    c = cache_on(0, watch)
    busy, mixed = set(), []

    def library(owner):
        def call(*args):
            if owner in busy:
                mixed.append(owner)
            busy.add(owner)
            time.sleep(0.002)
            busy.discard(owner)
            return moe.MOE_OK
        return call

    class Lib:
        def __getattr__(self, name):
            return (lambda *x: 256) if name.endswith("_bytes") else library("cache")
    a._prompt = a._decode = library("attention")
    c._lib = Lib()
    q, kv, i = Fake((3, 4, 64), torch.float32, 0), Fake((3, 2, 64), torch.float32, 0), lambda n: Fake((n,), torch.int32, 0)
    todo = [lambda: a.prompt(q, kv, kv, i(2), out=q), lambda: a.decode(q, c, i(3), out=q), lambda: c.resize(i(2), i(2)),
            lambda: c.write(kv, kv, i(2), i(3), i(2)), lambda: c.fork(i(2), i(2)), lambda: c.compact(i(1)),
            lambda: c.copy_pages(i(2), i(2)), c.clear]
    failed = []

    def run(k):
        try:
            for n in range(40):
                todo[(n + k) % len(todo)]()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=run, args=(k,)) for k in (0, 1, 3, 5)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and not mixed
