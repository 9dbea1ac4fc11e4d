"""Which workspace a call of Attention or KVCache gets. Needs no GPU: memory, streams and the library are stand-ins."""
import contextlib
import ctypes
import gc

import pytest
import torch

import sparse_mixture_experts_moe_gb300 as moe
from sparse_mixture_experts_moe_gb300 import _lib, attention
from sparse_mixture_experts_moe_gb300.attention import _Workspaces


BAD = moe.MOE_ERR_DEVICE_CHECK


class Memory:
    """A device tensor's place: `live` counts the ones that somebody still holds."""
    live, made = 0, 0

    def __init__(self, nbytes, device):
        Memory.live += 1
        Memory.made += 1
        self.nbytes, self.device = nbytes, device
        self.address = Memory.made << 40
        self.header = [0] * max(256, min(nbytes, 1 << 16))  # the bytes of its headers

    def __del__(self):
        Memory.live -= 1

    def data_ptr(self):
        return self.address

    def numel(self):
        return self.nbytes

    def __getitem__(self, part):
        return Part(self, part)


class Part:
    def __init__(self, memory, part):
        self.memory, self.part, self.device = memory, part, memory.device

    def copy_(self, other):
        self.memory.header[self.part] = other.memory.header[other.part]


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle

    def synchronize(self):
        pass


class Lib:
    """The library's calls that workspaces make."""

    def __init__(self):
        self.recording = {}  # stream -> number of the recording
        self.prepared = []
        self.mode, self.torch_records = 0, True

    def moe_stream_capture_id(self, stream):
        return self.recording.get(stream, 0)

    def moe_private_stream(self, stream):
        stream._obj.value = 0xABC0
        return moe.MOE_OK

    def moe_thread_capture_mode(self, mode):
        self.mode, was = mode, self.mode
        return was

    def init(self, ptr, nbytes, stream):
        assert self.mode == (2 if stream == 0xABC0 else 0)
        self.prepared.append((ptr, nbytes, stream))
        return moe.MOE_OK


def read_status(ws, stream=None):
    """moe_get_device_status on a stand-in: the header's first two places, cleared."""
    memory, at = (ws.memory, ws.part.start) if isinstance(ws, Part) else (ws, 0)
    got = tuple(memory.header[at:at + 2])
    memory.header[at:at + 2] = [0, 0]
    return got


def failed(memory, n):
    return [i for i in range(n) if memory.header[256 * i] != 0]


def fail(ws, row):
    """What a call on a workspace (or a recorded call on its header) leaves behind."""
    at = ws[2] - ws[0].address
    ws[0].header[at:at + 2] = [BAD, row]


@pytest.fixture
def world(monkeypatch):
    """A workspace pool on stand-ins, with the library and the devices that were selected."""
    lib, selected = Lib(), [0]

    @contextlib.contextmanager
    def device(d):
        selected.append(torch.device("cuda", d).index if isinstance(d, int) else d.index)
        yield
        selected.pop()

    monkeypatch.setattr(torch, "empty", lambda n, dtype=None, device=None: Memory(n, device))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda dev=None: None)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(_lib, "get_device_status", read_status)
    monkeypatch.setattr(attention, "_private_streams", {})
    monkeypatch.setattr(attention, "_kept", [])
    monkeypatch.setattr(attention, "_failed", failed)
    monkeypatch.setattr(attention, "_pooled_recording", (0, False))
    monkeypatch.setattr(attention, "_graph_owns", lambda t: lib.torch_records)
    pool = _Workspaces(lib, lib.init)
    return pool, lib, selected


def test_a_stream_keeps_its_workspace(world):
    pool, lib, _ = world
    a = pool.get(0, 1000, 0)
    assert pool.get(0, 1000, 0) == a and pool.get(0, 500, 0) == a
    b = pool.get(7, 1000, 0)
    assert b[2] != a[2] and pool.get(7, 800, 0) == b
    assert [p[0] for p in lib.prepared] == [a[2], b[2]]


def test_devices_do_not_share_workspaces(world):
    """The default stream has the same handle on every device."""
    pool, lib, _ = world
    a, b = pool.get(0, 1000, 0), pool.get(0, 1000, 1)
    assert a[2] != b[2] and (a[0].device.index, b[0].device.index) == (0, 1)
    assert pool.get(0, 1000, 0) == a and pool.get(0, 1000, 1) == b
    lib.recording[9] = 5
    c, d = pool.get(9, 1000, 0), pool.get(9, 1000, 1)
    assert len({x[2] for x in (a, b, c, d)}) == 4


def test_workspaces_are_prepared_and_read_on_their_device(world, monkeypatch):
    pool, lib, selected = world
    where = []
    monkeypatch.setattr(pool, "_init", lambda *a: where.append(("init", selected[-1])) or moe.MOE_OK)
    monkeypatch.setattr(_lib, "get_device_status", lambda ws, stream=None: where.append((ws.device.index, selected[-1])) or (moe.MOE_OK, 0))
    for dev in (0, 1, 3):
        pool.get(0, 1000, dev)
    assert pool.status() == (moe.MOE_OK, 0)
    assert where == [("init", 0), ("init", 1), ("init", 3), (0, 0), (1, 1), (3, 3)]


@pytest.mark.parametrize("stream", [0, 7])
def test_an_error_is_not_lost_when_a_workspace_grows(world, stream):
    pool, lib, _ = world
    fail(pool.get(stream, 1000, 0), 5)
    pool.get(stream, 2000, 0)
    pool.get(stream, 9000, 0)
    assert pool.status() == (BAD, 5)
    assert pool.status() == (moe.MOE_OK, 0)


def test_errors_of_all_workspaces_of_a_recording_are_read(world):
    """A graph goes on using the smaller workspace that its first calls recorded."""
    pool, lib, _ = world
    lib.recording[3] = 11
    small, large = pool.get(3, 1000, 0), pool.get(3, 5000, 0)
    lib.recording.clear()
    for ws, row in ((small, 4), (large, 6), (small, 8)):
        fail(ws, row)
        assert pool.status() == (BAD, row)
        assert pool.status() == (moe.MOE_OK, 0)


@pytest.mark.parametrize("stream", [0, 7])
def test_replaced_workspaces_are_given_back(world, stream):
    """A batch that grows by one sequence at a time keeps one workspace, and seldom makes a new one."""
    pool, lib, _ = world
    live, made = Memory.live, Memory.made
    for n in range(1, 257):
        assert pool.get(stream, 1000 + 100 * n, 0)[1] >= 1000 + 100 * n
    assert Memory.live - live == 1
    assert Memory.made - made <= 10


@pytest.mark.parametrize("torch_records", [True, False])
def test_living_graphs_share_nothing(world, torch_records):
    pool, lib, _ = world
    lib.torch_records = torch_records
    seen, scratch = set(), []
    for n in range(1, 101):  # more than one piece of headers
        lib.recording.update({3: n, 4: n})  # two streams of a recording
        for s in (3, 4):
            ws = pool.get(s, 1000, 0)
            assert ws[1] == 256 and ws[4] >= 744 and pool.get(s, 500, 0)[2] == ws[2]
            seen.add(ws[2])
            scratch.append(ws[5])
    lib.recording.clear()
    assert len(seen) == len(pool._recorded) == 200
    assert len({t.address for t in scratch}) == 200


def test_what_torchs_graphs_use_is_theirs_alone(world):
    """Scratch memory of the graph's own is not held beyond the call."""
    pool, lib, _ = world
    live = Memory.live
    for n in range(1, 129):
        lib.recording[3] = n
        pool.get(3, 1 << 20, 0)
    assert Memory.live - live == 2  # the headers


def test_what_other_recordings_use_is_kept(world):
    pool, lib, _ = world
    lib.torch_records = False
    live = Memory.live
    lib.recording[3] = 1
    at = pool.get(3, 1 << 20, 0)[3]
    del pool
    gc.collect()
    assert Memory.live - live == 2 and at in [t.address for t in attention._kept]


def test_what_a_capture_uses_is_kept_with_its_graph(world):
    pool, lib, _ = world
    live = Memory.live
    capture = _lib.GraphCapture()
    _lib.GraphCapture._now[77] = capture
    try:
        lib.recording[3] = 77
        a, b, c = (pool.get(3, n, 0) for n in (5000, 4000, 9000))
        assert a[3] == b[3] and c[3] != a[3]
    finally:
        del _lib.GraphCapture._now[77]
    assert {id(t) for t in capture._keep} == {id(a[5]), id(c[5])}
    del a, b, c, capture
    gc.collect()
    assert Memory.live - live == 1  # the headers


def test_a_cache_has_one_workspace(world):
    _, lib, _ = world
    pool = attention._CacheWorkspace(lib, lib.init)
    a = pool.get(0, 3000, 0)
    lib.recording[5] = 9
    assert pool.get(7, 3000, 0) is a and pool.get(5, 3000, 0) is a and len(lib.prepared) == 1
    fail(a, 3)
    assert pool.status() == (BAD, 3) and pool.status() == (moe.MOE_OK, 0)
    other = attention._CacheWorkspace(lib, lib.init)
    b = other.get(5, 3000, 0)  # made while recording: prepared beside it
    assert lib.prepared[-1][2] == 0xABC0 and other.get(0, 3000, 0) is b


@pytest.mark.parametrize("dev", [0, 1])
def test_a_recording_on_a_used_stream_shares_nothing_with_it(world, dev):
    """The graph may run on any stream, and beside further calls on this one."""
    pool, lib, _ = world
    eager = pool.get(6, 1000, dev)
    lib.recording[6] = 5
    first = pool.get(6, 1000, dev, 5)
    lib.recording[6] = 8
    second = pool.get(6, 1000, dev, 8)
    assert len({eager[2], first[2], second[2]}) == 3
    lib.recording.clear()
    assert pool.get(6, 1000, dev, 0) is eager


@pytest.mark.parametrize("pool,owned", [((0, 0), False), ((0, 7), True), ((3, 0), True), (None, False)])
def test_whose_memory_it_is(monkeypatch, pool, owned):
    """Only memory of a graph's own pool is left to the graph; an allocator that cannot say has none."""
    t = Memory(64, None)

    def snapshot():
        if pool is None:
            raise RuntimeError("no record")
        return [dict(address=t.address - 4096, total_size=4096, segment_pool_id=(9, 9)),
                dict(address=t.address - 512, total_size=2048, segment_pool_id=pool)]
    monkeypatch.setattr(torch.cuda, "memory_snapshot", snapshot)
    assert attention._graph_owns(t) is owned
