"""Attention and the paged key/value cache around the MoE layer (moe_attention_*, moe_cache_* of include/moe.h).

    attn = Attention(heads=32, kv_heads=8, head_dim=128, dtype=torch.bfloat16)
    out = attn.prompt(q, k, v, offsets)               # packed prompts, causal
    cache = KVCache.create(n_layers, n_pages, page_size, n_slots, max_len, kv_heads=8, head_dim=128,
                           dtype=torch.bfloat16, device="cuda")
    cache.resize(slots, new_lens)                     # pages for the new positions (0 frees a slot)
    cache.write(k, v, slots, offsets, pos, layer=l)   # their keys and values, once per layer
    out = attn.decode(q, cache, slots, layer=l, shared_len=n)   # one token a sequence
    cache.fork(src, dst)                              # samples of one sequence share its full pages

The tensors are on the current device. Everything is enqueued on the current stream, or on `stream`; nothing
synchronises. Calls can be recorded into a graph (torch.cuda.graph, GraphCapture), which keeps the workspace that they use;
an error that a replay records stays until device_status() reads it. Index tensors (offsets, slots, lengths, positions)
are int32 CUDA tensors. Arguments are marshalled and checked here; the work is done by the library's kernels.
"""
from __future__ import annotations

import contextlib
import ctypes

from . import _lib
from ._lib import MOE_ERR_INVALID_ARG, MOE_OK, MoeError, _check, _ptr, _stream


_HEADER = 256           # bytes of a workspace's header
_RELAXED = 2            # cudaStreamCaptureModeRelaxed
_SPLIT_KEYS = 1024      # moe_attention_prompt uses no more than the header below this many keys


class _Cache(ctypes.Structure):
    """moe_kv_cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("table", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("refs", ctypes.c_void_p), ("n_layers", ctypes.c_int), ("n_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("n_slots", ctypes.c_int), ("table_width", ctypes.c_int),
                ("H_kv", ctypes.c_int), ("D", ctypes.c_int), ("dt", ctypes.c_int), ("plan", ctypes.c_void_p)]


# The checks below run on every call, where a decode step's kernels take a few microseconds: each looks at a
# tensor's attributes once and formats a message only when it refuses.
def _heads(t, name, heads, dim, dtype, dev):
    """Checks a [T, heads, dim] tensor on CUDA device `dev` whose heads are dense within a token; returns (T, token
    stride)."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"moe: expected {name} [T, {heads}, {dim}] in {dtype} on cuda:{dev}, got {tuple(shape)} in "
                         f"{t.dtype} on {t.device}")
    st, sh, sd = t.stride()
    if sd != 1 or (sh != dim and heads > 1):
        raise ValueError(f"moe: {name} must have dense heads within a token (strides {t.stride()})")
    # a single token's stride means nothing: any valid one will do
    T = shape[0]
    return T, (st if T > 1 else heads * dim)


def _ints(t, name, n, dev, i32):
    """Checks an int32 index tensor of n entries (None: any number) on CUDA device `dev`; returns its length."""
    shape = t.shape
    if len(shape) != 1 or t.dtype is not i32 or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"moe: {name} must be a contiguous one-dimensional int32 tensor on cuda:{dev}")
    if n is not None and shape[0] != n:
        raise ValueError(f"moe: {name} has {shape[0]} entries; the call needs {n}")
    return shape[0]


class _Bound:
    """What the classes below look up once, not in every call."""

    def __init__(self):
        import torch
        self._lib = _lib.lib()
        self._i32 = torch.int32
        self._f32 = torch.float32
        self._empty, self._empty_like = torch.empty, torch.empty_like
        # the current stream's handle alone, without a stream object around it
        self._raw_stream = torch._C._cuda_getCurrentRawStream
        self._current_device = torch._C._cuda_getDevice
        self._ws = _Workspaces(self._lib, self._init_workspace)

    def _init_workspace(self, ptr, nbytes, stream):
        return self._lib.moe_workspace_init(ptr, nbytes, stream)

    def _stream_on(self, dev, stream):
        """The stream's handle for a call on tensors of CUDA device `dev`. Kernels run on the current device."""
        if self._current_device() != dev:
            raise ValueError(f"moe: the tensors are on cuda:{dev}, which is not the current device (torch.cuda.device)")
        return self._raw_stream(dev) if stream is None else _stream(stream)

    def device_status(self):
        """(status, detail) of the first device-side error since the last call; synchronises."""
        return self._ws.status()


class _Recorded:
    """A workspace that recorded calls use, and whether their graph is gone."""

    def __init__(self, lib, stream, key, ws):
        self._lib, self.key, self.ws = lib, key, ws
        self._ended = ctypes.POINTER(ctypes.c_int)()
        lib.moe_capture_watch(stream, ctypes.byref(self._ended))  # (without a watch: kept for good)

    def gone(self):
        return bool(self._ended) and self._ended[0] != 0

    def __del__(self):
        if self._ended:
            self._lib.moe_capture_watch_free(self._ended)


_in_graphs = set()     # _Recorded of all objects: a graph may outlive the Attention or KVCache whose calls it recorded
_private_streams = {}  # device -> a stream on which recordings' workspaces are allocated and prepared


def _private_stream(lib, dev):
    s = _private_streams.get(dev)
    if s is None:
        p = ctypes.c_void_p()
        _check(lib.moe_private_stream(ctypes.byref(p)), "moe_private_stream")
        s = _private_streams[dev] = p.value
    return s


def _size_class(n):
    """The next power of two, or three quarters of one: few sizes, so that a workspace that a graph leaves fits another."""
    p = 1 << max(n - 1, 1).bit_length()
    return p * 3 // 4 if n <= p * 3 // 4 else p


class _Workspaces:
    """Prepared workspaces, one for each stream (of each device) that calls arrive on, so that calls on different streams
    never share scratch memory, and one for each graph recording (and stream of it), which nothing else uses while the
    graph lives, however late and on whatever stream it runs. It is prepared beside the recording, once, so an error that a
    replay records stays until it is read; when the graph is gone another recording gets it. (A recording on a stream that
    calls have used before takes that stream's: its replays are to be ordered with further calls there.) A stream's is
    given back when a larger one replaces it."""

    def __init__(self, lib, init):
        self._lib, self._init = lib, init
        self._of = {}        # stream -> (tensor, bytes, address); (stream, device) on others than the first device,
                             # as the default stream has one handle for all of them
        self._recorded = {}  # (stream, recording, device) -> the same
        self._graphs = []    # _Recorded: of these, and those that larger ones replaced, which their graph uses too
        self._idle = []      # (device, the same): their graph is gone

    def get(self, stream, nbytes, dev):
        ws = self._of.get(stream if dev == 0 else (stream, dev))
        return ws if ws is not None and ws[1] >= nbytes else self._make(stream, nbytes, dev)

    def _make(self, stream, nbytes, dev):
        import torch
        recording = self._lib.moe_stream_capture_id(stream)
        if recording:
            return self._make_recorded(stream, recording, nbytes, dev)
        key = stream if dev == 0 else (stream, dev)
        old = self._of.get(key)
        if old is not None:
            if old[1] >= nbytes:
                return old
            nbytes = max(nbytes, old[1] * 3 // 2)  # a batch that grows one by one
        current = torch.cuda.current_stream(dev).cuda_stream == (stream or 0)
        # Memory of the stream's own: what was enqueued there is done with it before the next call that gets it runs, so the
        # workspace that this one replaces can be given back at once.
        with contextlib.nullcontext() if current else torch.cuda.stream(torch.cuda.ExternalStream(stream or 0, device=dev)):
            t = torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", dev))
            ws = (t, nbytes, t.data_ptr())
            with torch.cuda.device(dev):
                _check(self._init(ws[2], nbytes, stream), "workspace_init")
            if old is not None:  # an error that nobody has read yet
                t[:_HEADER].copy_(old[0][:_HEADER])
        self._of[key] = ws
        return ws

    def _make_recorded(self, stream, recording, nbytes, dev):
        import torch
        key = (stream, recording, dev)
        ws = self._recorded.get(key)
        if ws is not None and ws[1] >= nbytes:
            return ws
        self._sweep()
        fit = min((w for w in self._idle if w[0] == dev and w[1][1] >= nbytes), key=lambda w: w[1][1], default=None)
        if fit is not None:
            self._idle.remove(fit)
            ws = fit[1]
        else:
            # not the recording's memory, which its graph may use for other things before and after these calls
            nbytes, private = _size_class(nbytes), _private_stream(self._lib, dev)
            beside = torch.cuda.ExternalStream(private, device=dev)
            mode = self._lib.moe_thread_capture_mode(_RELAXED)  # this thread's other calls are to allocate and wait
            try:
                with torch.cuda.device(dev), torch.cuda.stream(beside):
                    t = torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", dev))
                    ws = (t, nbytes, t.data_ptr())
                    _check(self._init(ws[2], nbytes, private), "workspace_init")
                    beside.synchronize()
            finally:
                self._lib.moe_thread_capture_mode(mode)
        held = _Recorded(self._lib, stream, key, ws)
        self._graphs.append(held)
        _in_graphs.add(held)
        self._recorded[key] = ws
        return ws

    def _sweep(self):
        """Takes back what graphs that are gone have used."""
        _in_graphs.difference_update([r for r in _in_graphs if r.gone()])
        for r in [r for r in self._graphs if r.gone()]:
            self._graphs.remove(r)
            if self._recorded.get(r.key) is r.ws:
                del self._recorded[r.key]
            self._idle.append((r.key[2], r.ws))

    def status(self):
        """(status, detail) of the first device-side error of any of them; clears it."""
        import torch
        for key, ws in self._of.items():
            with torch.cuda.device(ws[0].device):
                st, detail = _lib.get_device_status(ws[0], key[0] if type(key) is tuple else key)
            if st != MOE_OK:
                return st, detail
        recorded = [r.ws for r in self._graphs] + [w[1] for w in self._idle]
        for dev in {ws[0].device for ws in recorded}:
            torch.cuda.synchronize(dev)
        for ws in recorded:
            with torch.cuda.device(ws[0].device):
                st, detail = _lib.get_device_status(ws[0])
            if st != MOE_OK:
                return st, detail
        return MOE_OK, 0


class KVCache(_Bound):
    """A paged key/value cache over tensors that the caller owns: k, v [layers, pages, kv_heads, page_size,
    head_dim] (bf16 or fp32), table [slots, width], lens [slots], refs [pages] (int32). KVCache.create
    allocates an empty one."""

    def __init__(self, k, v, table, lens, refs):
        import torch
        if k.dim() != 5 or k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("KVCache: expected k and v [layers, pages, kv_heads, page_size, head_dim] alike")
        if table.dim() != 2 or lens.shape != table.shape[:1] or refs.shape != k.shape[1:2]:
            raise ValueError("KVCache: expected table [slots, width], lens [slots], refs [pages]")
        for name, t in (("table", table), ("lens", lens), ("refs", refs)):
            if t.dtype != torch.int32:
                raise ValueError(f"KVCache: {name} must be int32")
        if any(t.device != k.device for t in (v, table, lens, refs)):
            raise ValueError("KVCache: all tensors must be on one device")
        self.k, self.v, self.table, self.lens, self.refs = k, v, table, lens, refs
        self.n_layers, self.n_pages, self.kv_heads, self.page_size, self.head_dim = (int(x) for x in k.shape)
        self.n_slots, self.width = (int(x) for x in table.shape)
        self.dtype, self.device = k.dtype, k.device
        self.dt = _lib.dtype_code(k)
        self._c = _Cache(_ptr(k), _ptr(v), _ptr(table), _ptr(lens), _ptr(refs), self.n_layers, self.n_pages,
                         self.page_size, self.n_slots, self.width, self.kv_heads, self.head_dim, self.dt)
        self._ref = ctypes.addressof(self._c)
        super().__init__()
        self._bytes = int(self._lib.moe_cache_workspace_bytes(self._ref))
        if self._bytes == 0:
            raise MoeError(MOE_ERR_INVALID_ARG, "moe_cache_workspace_bytes")
        self._dev = k.get_device()
        self._key = (self.kv_heads, self.head_dim, self.dtype)
        n = int(self._lib.moe_cache_plan_bytes())
        self._plan = ctypes.create_string_buffer(n)
        _check(self._lib.moe_cache_plan(self._ref, ctypes.addressof(self._plan), n), "moe_cache_plan")
        self._c.plan = ctypes.addressof(self._plan)

    @classmethod
    def create(cls, n_layers, n_pages, page_size, n_slots, max_len, kv_heads, head_dim, dtype, device="cuda"):
        """An empty cache: n_pages pages of page_size positions, n_slots sequences of at most max_len."""
        import torch
        width = max(1, -(-max_len // page_size))
        k = torch.empty((n_layers, n_pages, kv_heads, page_size, head_dim), dtype=dtype, device=device)
        i32 = dict(dtype=torch.int32, device=device)
        return cls(k, torch.empty_like(k), torch.full((n_slots, width), -1, **i32), torch.zeros(n_slots, **i32),
                   torch.zeros(n_pages, **i32))

    def _init_workspace(self, ptr, nbytes, stream):
        return self._lib.moe_cache_workspace_init(self._ref, ptr, nbytes, stream)

    def _workspace(self, stream):
        return self._ws.get(stream, self._bytes, self._dev)

    def clear(self, stream=None):
        """Empties every slot and frees every page."""
        s = self._stream_on(self._dev, stream)
        _check(self._lib.moe_cache_clear(self._ref, s), "moe_cache_clear")

    def resize(self, slots, new_lens, stream=None):
        """Slot slots[i] gets length new_lens[i]: pages are released (0 frees the slot) or allocated."""
        n = _ints(slots, "slots", None, self._dev, self._i32)
        _ints(new_lens, "new_lens", n, self._dev, self._i32)
        s = self._stream_on(self._dev, stream)
        ws = self._workspace(s)
        _check(self._lib.moe_cache_resize(self._ref, slots.data_ptr(), new_lens.data_ptr(), n, ws[2], ws[1], s),
               "moe_cache_resize")

    def write(self, k, v, slots, offsets, pos, layer=0, stream=None):
        """Tokens offsets[i] .. offsets[i+1]-1 of k, v [total, kv_heads, head_dim] become positions pos[i], pos[i]+1,
        ... of slot slots[i] in one layer."""
        total, ks = _heads(k, "k", self.kv_heads, self.head_dim, self.dtype, self._dev)
        tv, vs = _heads(v, "v", self.kv_heads, self.head_dim, self.dtype, self._dev)
        if tv != total:
            raise ValueError(f"moe: k has {total} tokens, v has {tv}")
        n = _ints(slots, "slots", None, self._dev, self._i32)
        _ints(offsets, "offsets", n + 1, self._dev, self._i32)
        _ints(pos, "pos", n, self._dev, self._i32)
        s = self._stream_on(self._dev, stream)
        ws = self._workspace(s)
        _check(self._lib.moe_cache_write(self._ref, layer, slots.data_ptr(), offsets.data_ptr(), pos.data_ptr(), n, total,
                                         k.data_ptr(), v.data_ptr(), ks, vs, ws[2], ws[1], s), "moe_cache_write")

    def fork(self, src, dst, stream=None):
        """Slot dst[i] becomes a copy of slot src[i], sharing its full pages; what dst[i] held is released."""
        n = _ints(src, "src", None, self._dev, self._i32)
        _ints(dst, "dst", n, self._dev, self._i32)
        s = self._stream_on(self._dev, stream)
        ws = self._workspace(s)
        _check(self._lib.moe_cache_fork(self._ref, src.data_ptr(), dst.data_ptr(), n, ws[2], ws[1], s), "moe_cache_fork")

    def compact(self, n_live=None, stream=None):
        """Moves the pages in use to the pool's lowest page numbers; returns their number, a one-entry int32
        tensor (n_live, if given)."""
        if n_live is None:
            if stream is not None:
                raise ValueError("moe: pass n_live with an explicit stream")
            n_live = self._empty(1, dtype=self._i32, device=self.device)
        _ints(n_live, "n_live", 1, self._dev, self._i32)
        s = self._stream_on(self._dev, stream)
        ws = self._workspace(s)
        _check(self._lib.moe_cache_compact(self._ref, n_live.data_ptr(), ws[2], ws[1], s), "moe_cache_compact")
        return n_live

    def copy_pages(self, src, dst, stream=None):
        """Page dst[i] gets page src[i]'s contents in every layer."""
        n = _ints(src, "src", None, self._dev, self._i32)
        _ints(dst, "dst", n, self._dev, self._i32)
        s = self._stream_on(self._dev, stream)
        ws = self._workspace(s)
        _check(self._lib.moe_cache_copy_pages(self._ref, src.data_ptr(), dst.data_ptr(), n, ws[2], ws[1], s),
               "moe_cache_copy_pages")


class Attention(_Bound):
    """Attention of `heads` query heads over `kv_heads` key/value heads of head_dim elements. Holds a workspace."""

    def __init__(self, heads, kv_heads, head_dim, dtype, scale=None):
        import torch
        if dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"unsupported dtype {dtype}")
        self.heads, self.kv_heads, self.head_dim, self.dtype = int(heads), int(kv_heads), int(head_dim), dtype
        self.dt = _lib.MOE_DTYPE_BF16 if dtype == torch.bfloat16 else _lib.MOE_DTYPE_F32
        if (self.heads < 1 or self.kv_heads < 1 or self.heads % self.kv_heads or self.head_dim % 8
                or not 8 <= self.head_dim <= 256):
            raise ValueError("Attention: heads must be a multiple of kv_heads, head_dim a multiple of 8 from 8 to 256")
        self.scale = float(scale) if scale is not None else self.head_dim ** -0.5
        super().__init__()
        self._sized, self._sized_bytes = None, 0
        self._prompt_bytes = self._lib.moe_attention_prompt_workspace_bytes
        self._prompt, self._decode = self._lib.moe_attention_prompt, self._lib.moe_attention_decode
        self._key = (self.kv_heads, self.head_dim, self.dtype)
        self._need = {}

    def _workspace(self, stream, n, dev):
        need = self._need.get(n)
        if need is None:
            need = int(self._lib.moe_attention_workspace_bytes(n, self.heads, self.head_dim))
            if need == 0:
                raise MoeError(MOE_ERR_INVALID_ARG, "moe_attention_workspace_bytes")
            self._need[n] = need
        return self._ws.get(stream, need, dev)

    def _out(self, q, out, lse, stream, dev):
        if out is None:
            if stream is not None:  # a tensor made here belongs to the current stream
                raise ValueError("moe: pass out with an explicit stream")
            out = self._empty_like(q) if q.is_contiguous() else self._empty(q.shape, dtype=self.dtype, device=q.device)
            so = self.heads * self.head_dim
        else:
            to, so = _heads(out, "out", self.heads, self.head_dim, self.dtype, dev)
            if to != q.shape[0]:
                raise ValueError(f"moe: expected out {tuple(q.shape)}, got {tuple(out.shape)}")
        if lse is not None:
            if (lse.shape != q.shape[:2] or lse.dtype is not self._f32 or lse.get_device() != dev
                    or not lse.is_contiguous()):
                raise ValueError(f"moe: expected lse {tuple(q.shape[:2])}, float32, contiguous, on {q.device}")
        return out, so

    def prompt(self, q, k, v, q_offsets, kv_offsets=None, causal=True, out=None, lse=None, stream=None):
        """Attention over packed prompts: q [Tq, heads, head_dim], k and v [Tkv, kv_heads, head_dim]; sequence i has
        queries q_offsets[i] .. q_offsets[i+1]-1 and keys kv_offsets[i] .. kv_offsets[i+1]-1 (the same where
        kv_offsets is None). causal: the queries are the last positions of their sequence. Returns out like q;
        lse [Tq, heads] (float32, optional) receives the logarithms of the softmax sums."""
        dev = q.get_device()
        if dev < 0:
            raise ValueError(f"moe: q, k and v must be CUDA tensors (got one on {q.device})")
        Tq, qs = _heads(q, "q", self.heads, self.head_dim, self.dtype, dev)
        Tk, ks = _heads(k, "k", self.kv_heads, self.head_dim, self.dtype, dev)
        Tv, vs = _heads(v, "v", self.kv_heads, self.head_dim, self.dtype, dev)
        if Tv != Tk or (kv_offsets is None and Tk != Tq):
            raise ValueError(f"moe: k has {Tk} tokens, v has {Tv}, q has {Tq}")
        n = _ints(q_offsets, "q_offsets", None, dev, self._i32) - 1
        if n < 0:
            raise ValueError("moe: q_offsets has one entry more than there are sequences")
        if kv_offsets is not None:
            _ints(kv_offsets, "kv_offsets", n + 1, dev, self._i32)
        out, so = self._out(q, out, lse, stream, dev)
        s = self._stream_on(dev, stream)
        need = _HEADER
        if Tk >= _SPLIT_KEYS:
            if self._sized != (n, Tq, Tk, dev):  # the layers of a model call with the same sizes
                self._sized_bytes = self._prompt_bytes(n, Tq, Tk, self.heads, self.kv_heads, self.head_dim, self.dt)
                self._sized = (n, Tq, Tk, dev)
            need = self._sized_bytes
        ws = self._ws.get(s, need, dev)
        _check(self._prompt(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), q_offsets.data_ptr(),
            None if kv_offsets is None else kv_offsets.data_ptr(), n, Tq, Tk, self.heads, self.kv_heads, self.head_dim,
            qs, ks, vs, so, self.scale, _lib.ATTN_CAUSAL if causal else 0, self.dt, out.data_ptr(),
            None if lse is None else lse.data_ptr(), ws[2], ws[1], s), "moe_attention_prompt")
        return out

    def decode(self, q, cache, slots, layer=0, shared_len=0, out=None, lse=None, stream=None):
        """One token for each sequence: q [n, heads, head_dim] attends the positions of slot slots[i] of the cache.
        shared_len: how many first positions of all n slots are the same pages (a multiple of the page size),
        read once for the whole batch."""
        dev = cache._dev
        if cache._key != self._key:
            raise ValueError(f"moe: the cache holds {cache.kv_heads} heads of {cache.head_dim} in {cache.dtype}, the "
                             f"attention {self.kv_heads} of {self.head_dim} in {self.dtype}")
        n, qs = _heads(q, "q", self.heads, self.head_dim, self.dtype, dev)
        _ints(slots, "slots", n, dev, self._i32)
        out, so = self._out(q, out, lse, stream, dev)
        s = self._stream_on(dev, stream)
        ws = self._workspace(s, n, dev)
        _check(self._decode(cache._ref, layer, q.data_ptr(), slots.data_ptr(), n, self.heads, qs, so, shared_len, self.scale,
                            out.data_ptr(), None if lse is None else lse.data_ptr(), ws[2], ws[1], s),
               "moe_attention_decode")
        return out
