"""Which workspace a call of Attention or KVCache gets. Needs no GPU: memory, streams and the library are stand-ins."""
import contextlib
import ctypes
import gc

import pytest
import torch

import sparse_mixture_experts_moe_gb300 as moe
from sparse_mixture_experts_moe_gb300 import _lib, attention
from sparse_mixture_experts_moe_gb300.attention import _Workspaces


class Memory:
    """A device tensor's place: `live` counts the ones that somebody still holds."""
    live, made = 0, 0

    def __init__(self, nbytes, device):
        Memory.live += 1
        Memory.made += 1
        self.nbytes, self.device = nbytes, device
        self.address = Memory.made << 40
        self.header = [0] * 256  # the header's bytes

    def __del__(self):
        Memory.live -= 1

    def data_ptr(self):
        return self.address

    def __getitem__(self, part):
        return Part(self, part)


class Part:
    def __init__(self, memory, part):
        self.memory, self.part = memory, part

    def any(self):
        return any(self.memory.header[self.part])

    def copy_(self, other):
        self.memory.header[self.part] = other.memory.header[other.part]


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle

    def synchronize(self):
        pass

    def wait_stream(self, other):
        pass


class Lib:
    """The library's calls that workspaces make."""

    def __init__(self):
        self.recording = {}  # stream -> number of the recording
        self.prepared = []
        self.watches, self.freed, self.mode = {}, 0, 0

    def moe_stream_capture_id(self, stream):
        return self.recording.get(stream, 0)

    def moe_capture_watch(self, stream, ended):
        flag = ctypes.c_int(0)
        self.watches.setdefault(self.recording[stream], []).append(flag)
        ended._obj.contents = flag
        return moe.MOE_OK

    def moe_capture_watch_free(self, ended):
        self.freed += 1
        return moe.MOE_OK

    def moe_private_stream(self, stream):
        stream._obj.value = 0xABC0
        return moe.MOE_OK

    def moe_thread_capture_mode(self, mode):
        self.mode, was = mode, self.mode
        return was

    def gone(self, recording):
        """The recording's graph is destroyed."""
        for flag in self.watches.pop(recording):
            flag.value = 1

    def init(self, ptr, nbytes, stream):
        assert self.mode == (2 if stream == 0xABC0 else 0)
        self.prepared.append((ptr, nbytes, stream))
        return moe.MOE_OK


def read_status(ws, stream=None):
    """moe_get_device_status on a stand-in: the header's first two places, cleared."""
    got = tuple(ws.header[:2])
    ws.header[:2] = [0, 0]
    return got


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
    monkeypatch.setattr(attention, "_in_graphs", set())
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


BAD = moe.MOE_ERR_DEVICE_CHECK


@pytest.mark.parametrize("stream", [0, 7])
def test_an_error_is_not_lost_when_a_workspace_grows(world, stream):
    pool, lib, _ = world
    pool.get(stream, 1000, 0)[0].header[:2] = [BAD, 5]
    pool.get(stream, 2000, 0)
    pool.get(stream, 9000, 0)
    assert pool.status() == (BAD, 5)
    assert pool.status() == (moe.MOE_OK, 0)


def test_errors_of_all_workspaces_of_a_recording_are_read(world):
    """A graph goes on using the smaller workspace that its first calls recorded."""
    pool, lib, _ = world
    lib.recording[3] = 11
    small = pool.get(3, 1000, 0)
    large = pool.get(3, 5000, 0)
    assert small[2] != large[2]
    lib.recording.clear()
    for ws, row in ((small, 4), (large, 6), (small, 8)):
        ws[0].header[:2] = [BAD, row]
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


def test_recordings_whose_graph_is_gone_leave_their_workspace_to_the_next(world):
    pool, lib, _ = world
    live = Memory.live
    for n in range(1, 200):
        lib.recording[3] = n
        assert pool.get(3, 1000 + n, 0)[1] >= 1000 + n
        lib.recording.clear()
        lib.gone(n)
    assert Memory.live - live <= 2 and len(pool._recorded) <= 1
    assert lib.freed >= 190


def test_living_graphs_share_no_workspace(world):
    pool, lib, _ = world
    seen = set()
    for n in range(1, 9):
        lib.recording[3] = n
        a, b = pool.get(3, 1000, 0), pool.get(3, 1000, 0)
        assert a is b
        lib.recording[4] = n  # another stream of the same recording
        seen |= {a[2], pool.get(4, 1000, 0)[2]}
        lib.recording.clear()
    assert len(seen) == 16
    lib.gone(5)
    lib.recording[3] = 20
    assert pool.get(3, 1000, 0)[2] in seen
    lib.recording.clear()
    assert len({w[2] for w in pool._recorded.values()}) == len(pool._recorded) == 15


def test_an_error_of_a_graph_that_is_gone_is_read(world):
    pool, lib, _ = world
    lib.recording[3] = 1
    pool.get(3, 1000, 0)[0].header[:2] = [BAD, 9]
    lib.recording.clear()
    lib.gone(1)
    lib.recording[3] = 2
    pool.get(3, 1000, 0)
    lib.recording.clear()
    assert pool.status() == (BAD, 9) and pool.status() == (moe.MOE_OK, 0)


def test_a_graph_keeps_its_workspace_when_the_object_is_gone(world):
    pool, lib, _ = world
    live = Memory.live
    other = _Workspaces(lib, lib.init)
    lib.recording[3] = 1
    other.get(3, 1000, 0)
    lib.recording.clear()
    del other
    gc.collect()
    assert Memory.live - live == 1
    lib.gone(1)
    lib.recording[3] = 2
    pool.get(3, 1000, 0)  # any other recording finds that it is over
    gc.collect()
    assert Memory.live - live == 1
