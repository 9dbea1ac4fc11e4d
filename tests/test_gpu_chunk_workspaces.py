"""Workspaces, streams and graphs of Attention.chunk, KVCache.append and Rotary.apply on the GPU."""
import threading

import pytest
import torch

import sparse_mixture_experts_moe_gb300 as moe
from attention_cases import i32, offsets, tensor
from test_gpu_attention_workspaces import record
from test_gpu_chunk import pool

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
BAD, OK = moe.MOE_ERR_DEVICE_CHECK, moe.MOE_OK
KINDS = [(BF16, 64), (BF16, 256), (F32, 64)]  # tcgen05, warp MMAs, CUDA cores


def setup(dtype=BF16, D=64, lens=(700, 90, 33), nq=(5, 40, 33), H=8, Hk=2):
    c, _ = pool(list(lens), 16, Hk, D, dtype, 3)
    q = tensor((sum(nq), H, D), 1, dtype, DEV)
    return moe.Attention(H, Hk, D, dtype), c, q, i32(range(len(nq)), DEV), i32(offsets(nq), DEV)


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("kind", ["torch", "moe"])
def test_graph_outlives_its_attention(kind, dtype, D):
    a, c, q, slots, offs = setup(dtype, D)
    out, want = torch.zeros_like(q), a.chunk(q, c, slots, offs).clone()
    g, replay = record(kind, lambda s: a.chunk(q, c, slots, offs, out=out, stream=s), out)
    need = a._lib.moe_attention_chunk_workspace_bytes(c._ref, 3, len(q), 8)
    del a
    taken = [torch.full((need,), 255, dtype=torch.uint8, device=DEV) for _ in range(4)]  # whatever was given back
    for _ in range(3):
        out.zero_()
        replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert all((t == 255).all() for t in taken)


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("kind", ["torch", "moe"])
def test_two_graphs_and_eager_calls_share_nothing(kind, dtype, D):
    """Two graphs of one Attention replayed on two streams at once, with eager calls of other sizes on a third."""
    a, c, q, slots, offs = setup(dtype, D)
    outs = [torch.zeros_like(q) for _ in range(2)]
    want = a.chunk(q, c, slots, offs).clone()
    graphs = [record(kind, lambda s, o=o: a.chunk(q, c, slots, offs, out=o, stream=s), o) for o in outs]
    big = torch.cat([q] * 4)
    many, longer = i32([0, 1, 2] * 4, DEV), i32(offsets([5, 40, 33] * 4), DEV)
    more = a.chunk(big, c, many, longer).clone()
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    eager = []
    for _ in range(20):
        for (g, replay), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                replay() if kind == "torch" else replay(s.cuda_stream)
        with torch.cuda.stream(streams[2]):
            eager.append(a.chunk(big, c, many, longer))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs) and all(torch.equal(e, more) for e in eager)
    assert a.device_status() == (OK, 0)


@pytest.mark.parametrize("kind", ["torch", "moe"])
@pytest.mark.parametrize("dtype,D", KINDS)
def test_errors_stay_until_they_are_read(kind, dtype, D):
    a, c, q, slots, offs = setup(dtype, D)
    out = torch.zeros_like(q)
    g, replay = record(kind, lambda s: a.chunk(q, c, slots, offs, out=out, stream=s), out)
    good = slots.clone()
    slots[1] = 99
    replay()
    slots.copy_(good)
    replay()
    torch.cuda.synchronize()
    assert a.device_status() == (BAD, 1)
    replay()
    assert a.device_status() == (OK, 0)
    # and through a larger workspace
    slots[2] = -5
    a.chunk(q[:5], c, slots[2:], i32([0, 5], DEV))
    slots.copy_(good)
    a.chunk(torch.cat([q] * 3), c, torch.cat([slots] * 3), i32(offsets([5, 40, 33] * 3), DEV))
    assert a.device_status() == (BAD, 0) and a.device_status() == (OK, 0)


def test_calls_on_other_streams():
    """The kernels run on the stream they are given: what is enqueued there before is seen, what comes after waits."""
    a, c, q, slots, offs = setup()
    rope = moe.Rotary(64)
    pos = i32(range(len(q)), DEV)
    want_r = rope.apply(q, pos).clone()
    want = a.chunk(want_r, c, slots, offs).clone()
    k0, v0 = c.k.clone(), c.v.clone()
    x = tensor((len(q), 2, 64), 4, BF16, DEV)
    cache_pos = i32([695, 50, 0], DEV)  # the slots' last positions
    want_q = c.append(x, x, slots, offs, cache_pos, rope, q=q).clone()
    want_k = c.k.clone()
    c.k.copy_(k0)
    c.v.copy_(v0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    late, turned, out, qo = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q)
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        late.copy_(q)
    rope.apply(late, pos, out=turned, stream=s)
    a.chunk(turned, c, slots, offs, out=out, stream=s)
    c.append(x, x, slots, offs, cache_pos, rope, q=late, q_out=qo, stream=s)
    s.synchronize()
    assert torch.equal(turned, want_r) and torch.equal(out, want) and torch.equal(qo, want_q)
    assert torch.equal(c.k.nan_to_num(9.0), want_k.nan_to_num(9.0))
    assert c.device_status() == (OK, 0) and a.device_status() == (OK, 0)


@pytest.mark.parametrize("kind", ["torch", "moe"])
def test_a_recorded_step(kind):
    """A layer's step as one graph: queries and keys turned on the way into the cache, then attended; replayed on new
    contents it gives what the plain calls give, bit for bit."""
    H, Hk, D, n = 8, 2, 64, 5
    rope, a = moe.Rotary(D, scaling="linear", factor=2.0), moe.Attention(H, Hk, D, BF16)
    c, _ = pool([40, 17, 300, 1, 64], 16, Hk, D, BF16, 8)
    x, w = tensor((n, H + 2 * Hk, D), 5, BF16, DEV), tensor((D,), 6, BF16, DEV)
    slots, offs, pos = i32(range(n), DEV), i32(range(n + 1), DEV), c.lens - 1
    q, out = torch.empty((n, H, D), dtype=BF16, device=DEV), torch.empty((n, H, D), dtype=BF16, device=DEV)

    def step(stream=None):
        c.append(x[:, H:H + Hk], x[:, H + Hk:], slots, offs, pos, rope, q=x[:, :H], q_out=q, q_weight=w, k_weight=w, stream=stream)
        a.chunk(q, c, slots, offs, out=out, stream=stream)

    step()
    torch.cuda.synchronize()
    g, replay = record(kind, step, x, q, out)
    for seed in range(3):
        x.copy_(tensor(x.shape, 50 + seed, BF16, DEV))
        replay()
        torch.cuda.synchronize()
        got, k = out.clone(), c.k.clone()
        out.zero_()
        step()
        assert torch.equal(out, got) and torch.equal(c.k.nan_to_num(9.0), k.nan_to_num(9.0))
    assert c.device_status() == (OK, 0) and a.device_status() == (OK, 0)


def test_threads_share_an_attention_and_a_rotary():
    a, c, q, slots, offs = setup()
    rope, pos = moe.Rotary(64), i32(range(len(q)), DEV)
    sizes = [(q, slots, offs, pos), (q[:45], slots[:2], offs[:3], pos[:45]), (q[:5], slots[:1], offs[:2], pos[:5])]
    want = [a.chunk(rope.apply(x, p), c, s, o).clone() for x, s, o, p in sizes]
    torch.cuda.synchronize()
    failed = []

    def run(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for i in range(30):
                    x, s, o, p = sizes[(i + k) % 3]
                    got = a.chunk(rope.apply(x, p), c, s, o)
                    if not torch.equal(got, want[(i + k) % 3]):
                        failed.append((k, i))
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=run, args=(k,)) for k in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    assert a.device_status() == (OK, 0)


def test_padded_batch():
    """Sequences of no tokens at the end, and rows behind the last one: neither is touched."""
    for dtype, D in KINDS:
        a, c, q, _, _ = setup(dtype, D)
        slots, offs = i32([0, 1, 2, 0, 0, -7, 99], DEV), i32([0, 5, 45, 50, 50, 50, 50, 50], DEV)
        out = torch.full_like(q, 3.0)
        a.chunk(q, c, slots, offs, out=out)
        assert (out[50:] == 3).all() and torch.isfinite(out[:50]).all()
        want = a.chunk(q[:50], c, slots[:3], offs[:4])
        # (with more sequences the fp32 and long heads' keys may be cut elsewhere: same bounds, not the same bits)
        if D <= 128 and dtype == BF16:
            assert torch.equal(out[:50], want)
        assert a.device_status() == (OK, 0)  # slots of sequences without tokens are not looked at
