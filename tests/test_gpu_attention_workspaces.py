"""Workspaces of Attention on the GPU: what a larger one, a graph or a second thread does to them."""
import threading

import pytest
import torch

import sparse_mixture_experts_moe_gb300 as moe
from attention_cases import i32, tensor
from test_gpu_attention import BF16, DEV, F32, make_cache

pytestmark = pytest.mark.gpu
BAD, OK = moe.MOE_ERR_DEVICE_CHECK, moe.MOE_OK


def setup(n=12, H=8, Hk=2, D=64, shared=64, dtype=BF16):
    c, _ = make_cache([shared + 5 + 11 * i for i in range(n)], shared, 16, Hk, D, dtype)
    return moe.Attention(H, Hk, D, dtype), c, tensor((n, H, D), 1, dtype, DEV)


@pytest.mark.parametrize("own_stream", [False, True])
def test_an_error_is_not_lost_when_the_workspace_grows(own_stream):
    a, c, q = setup()
    s = torch.cuda.Stream() if own_stream else None
    out = torch.empty_like(q)
    torch.cuda.synchronize()

    def call(slots):
        a.decode(q[:len(slots)], c, i32(slots, DEV), out=out[:len(slots)], stream=s)

    call([0, 99])
    for n in (3, 5, 12):
        call(list(range(n)))
    assert a.device_status() == (BAD, 1)
    assert a.device_status() == (OK, 0)


@pytest.mark.parametrize("own_stream", [False, True])
def test_a_growing_batch_keeps_one_workspace(own_stream):
    a, c, q = setup(n=64, shared=32)
    s = torch.cuda.Stream() if own_stream else None
    want = a.decode(q, c, i32(range(64), DEV), shared_len=32)
    a = moe.Attention(8, 2, 64, BF16)
    out = torch.empty_like(q)
    slots = [i32(range(n), DEV) for n in range(65)]
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for n in range(1, 65):
        a.decode(q[:n], c, slots[n], shared_len=32, out=out[:n], stream=s)
    torch.cuda.synchronize()
    need = a._lib.moe_attention_workspace_bytes(64, 8, 64)
    assert torch.cuda.memory_allocated() - before <= 1.5 * need + 512
    assert torch.equal(out, want)
    assert a.device_status() == (OK, 0)


def record(kind, call, *keep):
    """A graph of call(stream), and how to replay it on a stream of its own choice."""
    if kind == "torch":
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(None)
        return g, g.replay
    with moe.GraphCapture(keep=keep) as cap:
        call(cap.stream)
    return cap, cap.graph.launch


@pytest.mark.parametrize("kind", ["torch", "moe"])
def test_recording_again_and_again_keeps_no_workspaces(kind):
    a, c, q = setup()
    slots, out = i32(range(12), DEV), torch.zeros_like(q)
    want = a.decode(q, c, slots, shared_len=64)
    need = a._lib.moe_attention_workspace_bytes(12, 8, 64)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for _ in range(12):
        g, replay = record(kind, lambda s: a.decode(q, c, slots, shared_len=64, out=out, stream=s), out)
        out.zero_()
        replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        del g, replay
        torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() - before < 1.5 * need
    assert a.device_status() == (OK, 0)


@pytest.mark.parametrize("kind", ["torch", "moe"])
def test_an_error_of_a_replay_stays_until_it_is_read(kind):
    a, c, q = setup()
    slots, out = i32(range(12), DEV), torch.zeros_like(q)
    good = slots.clone()
    g, replay = record(kind, lambda s: a.decode(q, c, slots, shared_len=64, out=out, stream=s), out)
    assert a.device_status() == (OK, 0)
    slots[7] = 99
    replay()
    slots.copy_(good)
    replay()
    torch.cuda.synchronize()
    assert a.device_status() == (BAD, 7)
    replay()
    assert a.device_status() == (OK, 0)


@pytest.mark.parametrize("kind", ["torch", "moe"])
def test_a_graph_outlives_the_attention_that_it_recorded(kind):
    a, c, q = setup()
    slots, out = i32(range(12), DEV), torch.zeros_like(q)
    want = a.decode(q, c, slots, shared_len=64).clone()
    g, replay = record(kind, lambda s: a.decode(q, c, slots, shared_len=64, out=out, stream=s), out)
    need = a._lib.moe_attention_workspace_bytes(12, 8, 64)
    del a
    taken = [torch.full((need,), 255, dtype=torch.uint8, device=DEV) for _ in range(6)]  # whatever was given back
    for _ in range(3):
        out.zero_()
        replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert all((t == 255).all() for t in taken)


def test_a_recording_over_two_streams():
    a, c, q = setup()
    slots, outs = i32(range(12), DEV), [torch.zeros_like(q) for _ in range(2)]
    want = a.decode(q, c, slots, shared_len=64)
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        a.decode(q, c, slots, shared_len=64, out=outs[0], stream=side)
        a.decode(q, c, slots, shared_len=64, out=outs[1])
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(20):
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
    assert a.device_status() == (OK, 0)


def test_graphs_of_one_attention_run_at_the_same_time():
    """Each has a header of its own, and scratch memory of its own; so have prompts that are split."""
    a, c, q = setup()
    slots, want = i32(range(12), DEV), None
    x, o, ko = tensor((2000, 12, 64), 2, BF16, DEV), i32([0, 16], DEV), i32([0, 2000], DEV)
    want = a.decode(q, c, slots, shared_len=64)
    long = a.prompt(x[:16, :8], x[:, 8:10], x[:, 10:], o, ko)
    graphs = []
    for kind in ("torch", "moe", "torch", "moe"):
        outs = [torch.empty_like(want), torch.empty_like(long)]

        def calls(s, outs=outs):
            a.decode(q, c, slots, shared_len=64, out=outs[0], stream=s)
            a.prompt(x[:16, :8], x[:, 8:10], x[:, 10:], o, ko, out=outs[1], stream=s)

        graphs.append((*record(kind, calls), outs, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(25):
        for _, replay, outs, s in graphs:
            with torch.cuda.stream(s):
                replay()
        assert torch.equal(a.decode(q, c, slots, shared_len=64), want)
    torch.cuda.synchronize()
    for _, _, outs, _ in graphs:
        assert torch.equal(outs[0], want) and torch.equal(outs[1], long)
    assert a.device_status() == (OK, 0)


def test_recordings_on_a_used_stream_run_beside_it():
    """Two graphs recorded on a stream that calls have used, replayed on other streams while calls go on there."""
    a, c, q = setup(n=40)
    slots = i32(range(40), DEV)
    want = a.decode(q, c, slots, shared_len=64)
    used = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(used):
        a.decode(q, c, slots, shared_len=64)
    graphs = []
    for _ in range(2):
        g, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=used):
            a.decode(q, c, slots, shared_len=64, out=out)
        graphs.append((g, out, torch.cuda.Stream()))
    assert len({w[2] for w in a._ws._recorded.values()} | {w[2] for w in a._ws._of.values()}) == 4
    torch.cuda.synchronize()
    for _ in range(30):
        for g, _, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(used):
            again = a.decode(q, c, slots, shared_len=64)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for _, o, _ in graphs) and torch.equal(again, want)
    assert a.device_status() == (OK, 0)


def test_scratch_memory_apart():
    """moe_attention_decode_ex with scratch memory elsewhere, that holds anything: the same result; too little is refused."""
    a, c, q = setup()
    slots, out = i32(range(12), DEV), torch.zeros_like(q)
    want = a.decode(q, c, slots, shared_len=64)
    need = a._lib.moe_attention_workspace_bytes(12, 8, 64) - 256
    head, scratch = torch.zeros(256, dtype=torch.uint8, device=DEV), torch.full((need,), 255, dtype=torch.uint8, device=DEV)

    def call(nbytes, at=None, head_bytes=256):
        return a._lib.moe_attention_decode_ex(
            c._ref, 0, q.data_ptr(), slots.data_ptr(), 12, 8, 512, 512, 64, 64 ** -0.5, out.data_ptr(), None, head.data_ptr(),
            head_bytes, scratch.data_ptr() if at is None else at, nbytes, torch.cuda.current_stream().cuda_stream)

    assert call(need) == moe.MOE_OK
    assert torch.equal(out, want)
    for bad in (call(need - 1), call(need, scratch.data_ptr() + 8), call(need, 0), call(0, 0), call(need, None, 255)):
        assert bad == moe.MOE_ERR_INVALID_ARG


def test_cache_calls_in_graphs_recorded_again_and_again():
    c = moe.KVCache.create(2, 40, 16, 6, 160, 2, 32, BF16, DEV)
    slots, lens = i32([0, 3], DEV), i32([40, 17], DEV)
    for n in range(6):
        g, replay = record("torch", lambda s: c.resize(slots, lens, stream=s))
        lens.copy_(i32([40 + n, 17 + 20 * n], DEV))
        replay()
        torch.cuda.synchronize()
        assert c.lens.tolist() == [40 + n, 0, 0, 17 + 20 * n, 0, 0]
        assert int((c.refs > 0).sum()) == -(-(40 + n) // 16) + -(-(17 + 20 * n) // 16)
        assert c.device_status() == (OK, 0)


def test_two_threads_use_one_attention_on_one_stream():
    a, c, q = setup(n=24, H=16, Hk=2, D=128)
    rows = [i32(range(n), DEV) for n in (24, 7)]
    want = [a.decode(q[:len(r)], c, r, shared_len=64) for r in rows]
    torch.cuda.synchronize()
    outs, failed = [[], []], []

    def run(k):
        try:
            for _ in range(300):
                outs[k].append(a.decode(q[:len(rows[k])], c, rows[k], shared_len=64))
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=run, args=(k,)) for k in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for k in (0, 1):
        assert sum(not torch.equal(o, want[k]) for o in outs[k]) == 0
    assert a.device_status() == (OK, 0)


def test_calls_on_the_default_stream_while_another_is_current():
    a, c, q = setup()
    slots, out = i32(range(12), DEV), torch.zeros_like(q)
    want = moe.Attention(8, 2, 64, BF16).decode(q, c, slots, shared_len=64)
    grown = i32([40] * 3, DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for n in (2, 12):
            a.decode(q[:n], c, slots[:n], shared_len=64, out=out[:n], stream=torch.cuda.default_stream())
        fresh = moe.KVCache.create(1, 20, 16, 3, 64, 2, 32, BF16, DEV)
        torch.cuda.synchronize()
        fresh.resize(i32([0, 1, 2], DEV), grown, stream=torch.cuda.default_stream())
        torch.cuda.synchronize()
    assert torch.equal(out, want) and fresh.lens.tolist() == [40] * 3
    assert a.device_status() == (OK, 0) and fresh.device_status() == (OK, 0)
