"""Workspaces of Attention on the GPU: what a larger one, a graph or a second thread does to them."""
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
    assert torch.cuda.memory_allocated() - before < 4.5 * need
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


def test_a_workspace_is_watched_as_long_as_its_graph_can_run():
    """Not given to another recording while an executable graph is there, and given back after it."""
    a, c, q = setup()
    slots, out = i32(range(12), DEV), torch.zeros_like(q)
    g, replay = record("moe", lambda s: a.decode(q, c, slots, out=out, stream=s), out)
    replay()
    torch.cuda.synchronize()
    a._ws._sweep()
    assert len(a._ws._graphs) == 1 and not a._ws._graphs[0].gone()
    g.graph.close()
    torch.cuda.synchronize()
    for _ in range(200):
        if a._ws._graphs[0].gone():
            break
        torch.cuda._sleep(100000)
        torch.cuda.synchronize()
    a._ws._sweep()
    assert a._ws._graphs == [] and len(a._ws._idle) == 1


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
