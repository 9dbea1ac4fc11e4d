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
synchronises. Calls can be recorded into a graph (torch.cuda.graph, GraphCapture); an error that a replay records
stays until device_status() reads it. Calls on one KVCache must not overlap in time, on whatever streams they are.
Threads may share an Attention; they enqueue their calls one after the other. Index tensors (offsets, slots, lengths,
positions) are int32 CUDA tensors. Arguments are marshalled and checked here; the work is done by the library's kernels.
"""
from __future__ import annotations

import contextlib
import ctypes
import threading

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
        self._current_device, self._many = torch._C._cuda_getDevice, torch.cuda.device_count() > 1
        # Calls enqueue several kernels that use one workspace; threads take turns.
        self._lock = threading.Lock()
        self._ws = self._spaces(self._lib, self._init_workspace)

    def _elsewhere(self, dev):
        raise ValueError(f"moe: the tensors are on cuda:{dev}, which is not the current device (torch.cuda.device)")

    def device_status(self):
        """(status, detail) of the first device-side error since the last call; synchronises."""
        with self._lock:
            return self._ws.status()


_private_streams = {}  # device -> a stream that nothing but the functions here uses
_kept = []             # memory that graphs may use, whatever becomes of the object whose calls they recorded
_pooled_recording = (0, False)


def _private_stream(lib, dev):
    import torch
    s = _private_streams.get(dev)
    if s is None:
        p = ctypes.c_void_p()
        _check(lib.moe_private_stream(ctypes.byref(p)), "moe_private_stream")
        s = _private_streams[dev] = torch.cuda.ExternalStream(p.value, device=dev)
    return s


@contextlib.contextmanager
def _beside(lib, dev):
    """A stream to allocate and prepare memory on while another stream of this thread is recording; waits for it."""
    import torch
    with torch.cuda.device(dev):
        s = _private_stream(lib, dev)
        mode = lib.moe_thread_capture_mode(_RELAXED)  # else allocating and waiting would break the recording off
        try:
            with torch.cuda.stream(s):
                yield s.cuda_stream
                s.synchronize()
        finally:
            lib.moe_thread_capture_mode(mode)


def _on(stream, dev):
    """`stream` as the current one, so that memory allocated meanwhile is that stream's."""
    import torch
    if torch.cuda.current_stream(dev).cuda_stream == (stream or 0):
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream or 0, device=dev))


def _bytes(n, dev):
    import torch
    return torch.empty(n, dtype=torch.uint8, device=torch.device("cuda", dev))


def _graph_owns(t):
    """Whether a tensor is memory of a graph's own (of torch's graphs), which no other program part gets."""
    import torch
    at = t.data_ptr()
    try:
        segments = torch.cuda.memory_snapshot()
    except RuntimeError:  # an allocator that keeps no such record
        return False
    return any(s["address"] <= at < s["address"] + s["total_size"] and tuple(s.get("segment_pool_id", (0, 0))) != (0, 0)
               for s in segments)


def _scratch(lib, stream, recording, nbytes, dev):
    """Scratch memory of a recorded call. Only the call itself uses it, so the graph may use it for other things too,
    but nothing else may while the graph lives: it is the graph's own memory if torch records the graph, and kept with
    the graph if GraphCapture does. Of other recordings nobody knows when the graph is gone."""
    global _pooled_recording
    if nbytes == 0:
        return None
    capture = _lib.GraphCapture.of(recording)
    if capture is None:
        pooled = _pooled_recording
        with _on(stream, dev):
            if pooled[0] != recording:
                pooled = _pooled_recording = (recording, _graph_owns(_bytes(1, dev)))
            if pooled[1]:
                return _bytes(nbytes, dev)
    t = capture.scratch.get(stream) if capture is not None else None
    if t is None or t.numel() < nbytes:
        with _beside(lib, dev):
            t = _bytes(nbytes, dev)
        if capture is not None:
            capture.scratch[stream] = t
            capture.hold(t)
        else:
            _kept.append(t)
    return t


def _failed(headers, n):
    """Which of a tensor's first n headers hold an error."""
    import torch
    words = headers.view(torch.int32)[:n * _HEADER // 4:_HEADER // 4].tolist()
    return [i for i, w in enumerate(words) if w != MOE_OK]


class _Workspaces:
    """Prepared workspaces, one for each stream (of each device) that calls arrive on, so that calls on different
    streams never share scratch memory. A stream's is given back when a larger one replaces it. Calls that are recorded
    get a header of their own for each recording (and stream of it), and scratch memory that is the graph's (_scratch),
    so that nothing else uses either while the graph lives, however late and on whatever stream it runs. Headers are
    prepared beside the recording, once, and kept for good, 256 bytes each: an error that a replay records stays until
    it is read."""

    _HEADERS = 64  # of one piece of memory

    def __init__(self, lib, init):
        self._lib, self._init = lib, init
        self._of = {}        # stream -> (tensor, bytes, address); (stream, device) on others than the first device,
                             # as the default stream has one handle for all of them
        self._recorded = {}  # (stream, recording, device) -> the same, a header
        self._headers = {}   # device -> [(tensor, how many of its headers are taken)]

    def get(self, stream, nbytes, dev, recording=None):
        """recording: the number of the recording that the call is part of, 0 for none (None: the library is asked)."""
        if recording is None:
            recording = self._lib.moe_stream_capture_id(stream)
        if recording:
            return self._make_recorded(stream, recording, nbytes, dev)
        ws = self._of.get(stream if dev == 0 else (stream, dev))
        return ws if ws is not None and ws[1] >= nbytes else self._make(stream, nbytes, dev)

    def _make(self, stream, nbytes, dev):
        import torch
        key = stream if dev == 0 else (stream, dev)
        old = self._of.get(key)
        if old is not None:
            nbytes = max(nbytes, old[1] * 3 // 2)  # a batch that grows one by one
        # Memory of the stream's own: what was enqueued there is done with it before the next call that gets it runs, so
        # the workspace that this one replaces can be given back at once.
        with _on(stream, dev):
            t = _bytes(nbytes, dev)
            ws = (t, nbytes, t.data_ptr())
            with torch.cuda.device(dev):
                _check(self._init(ws[2], nbytes, stream), "workspace_init")
            if old is not None:  # an error that nobody has read yet
                t[:_HEADER].copy_(old[0][:_HEADER])
        self._of[key] = ws
        return ws

    def _make_recorded(self, stream, recording, nbytes, dev):
        """(header's tensor, bytes, address, scratch memory's address, bytes, tensor)"""
        key = (stream, recording, dev)
        head = self._recorded.get(key)
        if head is None:
            rows = self._headers.setdefault(dev, [])
            with _beside(self._lib, dev) as s:
                if not rows or rows[-1][1] == self._HEADERS:
                    rows.append((_bytes(self._HEADERS * _HEADER, dev), 0))
                    _kept.append(rows[-1][0])
                t, n = rows[-1]
                at = t.data_ptr() + n * _HEADER
                _check(self._init(at, _HEADER, s), "workspace_init")
            rows[-1] = (t, n + 1)
            head = self._recorded[key] = (t, _HEADER, at)
        t = _scratch(self._lib, stream, recording, nbytes - _HEADER, dev)
        return (*head, None, 0, None) if t is None else (*head, t.data_ptr(), t.numel(), t)

    def status(self):
        """(status, detail) of the first device-side error of any of them; clears it."""
        import torch
        for key, ws in self._of.items():
            with torch.cuda.device(ws[0].device):
                st, detail = _lib.get_device_status(ws[0], key[0] if type(key) is tuple else key)
            if st != MOE_OK:
                return st, detail
        for dev, rows in self._headers.items():
            with torch.cuda.device(dev):
                torch.cuda.synchronize()
                for t, n in rows:
                    for i in _failed(t, n):
                        return _lib.get_device_status(t[i * _HEADER:(i + 1) * _HEADER])
        return MOE_OK, 0


class _CacheWorkspace:
    """The workspace of a KVCache: one for all streams and graphs, as calls on one cache do not overlap in time. A graph
    of such calls needs it as it needs the cache's tensors."""

    def __init__(self, lib, init):
        self._lib, self._init, self._ws = lib, init, None

    def get(self, stream, nbytes, dev):
        return self._ws or self._make(stream, nbytes, dev)

    def _make(self, stream, nbytes, dev):
        import torch
        if self._lib.moe_stream_capture_id(stream):
            with _beside(self._lib, dev) as s:
                t = _bytes(nbytes, dev)
                _check(self._init(t.data_ptr(), nbytes, s), "workspace_init")
        else:
            with _on(stream, dev), torch.cuda.device(dev):
                t = _bytes(nbytes, dev)
                _check(self._init(t.data_ptr(), nbytes, stream), "workspace_init")
        self._ws = (t, nbytes, t.data_ptr())
        return self._ws

    def status(self):
        """(status, detail) of the first device-side error; clears it."""
        import torch
        if self._ws is None:
            return MOE_OK, 0
        with torch.cuda.device(self._ws[0].device):
            torch.cuda.synchronize()
            return _lib.get_device_status(self._ws[0])


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

    _spaces = _CacheWorkspace

    def _init_workspace(self, ptr, nbytes, stream):
        return self._lib.moe_cache_workspace_init(self._ref, ptr, nbytes, stream)

    def _workspace(self, stream):
        return self._ws.get(stream, self._bytes, self._dev)

    def clear(self, stream=None):
        """Empties every slot and frees every page."""
        if self._many and self._current_device() != self._dev:  # kernels run on the current device
            self._elsewhere(self._dev)
        s = self._raw_stream(self._dev) if stream is None else _stream(stream)
        with self._lock:
            _check(self._lib.moe_cache_clear(self._ref, s), "moe_cache_clear")

    def resize(self, slots, new_lens, stream=None):
        """Slot slots[i] gets length new_lens[i]: pages are released (0 frees the slot) or allocated."""
        n = _ints(slots, "slots", None, self._dev, self._i32)
        _ints(new_lens, "new_lens", n, self._dev, self._i32)
        if self._many and self._current_device() != self._dev:  # kernels run on the current device
            self._elsewhere(self._dev)
        s = self._raw_stream(self._dev) if stream is None else _stream(stream)
        with self._lock:
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
        if self._many and self._current_device() != self._dev:  # kernels run on the current device
            self._elsewhere(self._dev)
        s = self._raw_stream(self._dev) if stream is None else _stream(stream)
        with self._lock:
            ws = self._workspace(s)
            _check(self._lib.moe_cache_write(self._ref, layer, slots.data_ptr(), offsets.data_ptr(), pos.data_ptr(), n,
                                             total, k.data_ptr(), v.data_ptr(), ks, vs, ws[2], ws[1], s), "moe_cache_write")

    def fork(self, src, dst, stream=None):
        """Slot dst[i] becomes a copy of slot src[i], sharing its full pages; what dst[i] held is released."""
        n = _ints(src, "src", None, self._dev, self._i32)
        _ints(dst, "dst", n, self._dev, self._i32)
        if self._many and self._current_device() != self._dev:  # kernels run on the current device
            self._elsewhere(self._dev)
        s = self._raw_stream(self._dev) if stream is None else _stream(stream)
        with self._lock:
            ws = self._workspace(s)
            _check(self._lib.moe_cache_fork(self._ref, src.data_ptr(), dst.data_ptr(), n, ws[2], ws[1], s),
                   "moe_cache_fork")

    def compact(self, n_live=None, stream=None):
        """Moves the pages in use to the pool's lowest page numbers; returns their number, a one-entry int32
        tensor (n_live, if given)."""
        if n_live is None:
            if stream is not None:
                raise ValueError("moe: pass n_live with an explicit stream")
            n_live = self._empty(1, dtype=self._i32, device=self.device)
        _ints(n_live, "n_live", 1, self._dev, self._i32)
        if self._many and self._current_device() != self._dev:  # kernels run on the current device
            self._elsewhere(self._dev)
        s = self._raw_stream(self._dev) if stream is None else _stream(stream)
        with self._lock:
            ws = self._workspace(s)
            _check(self._lib.moe_cache_compact(self._ref, n_live.data_ptr(), ws[2], ws[1], s), "moe_cache_compact")
        return n_live

    def copy_pages(self, src, dst, stream=None):
        """Page dst[i] gets page src[i]'s contents in every layer."""
        n = _ints(src, "src", None, self._dev, self._i32)
        _ints(dst, "dst", n, self._dev, self._i32)
        if self._many and self._current_device() != self._dev:  # kernels run on the current device
            self._elsewhere(self._dev)
        s = self._raw_stream(self._dev) if stream is None else _stream(stream)
        with self._lock:
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
        self._prompt_ex, self._decode_ex = self._lib.moe_attention_prompt_ex, self._lib.moe_attention_decode_ex
        self._capturing, self._recording = torch._C._cuda_isCurrentStreamCapturing, self._lib.moe_stream_capture_id
        self._key = (self.kv_heads, self.head_dim, self.dtype)
        self._need = {}
        self._of = self._ws._of

    _spaces = _Workspaces

    def _init_workspace(self, ptr, nbytes, stream):
        return self._lib.moe_workspace_init(ptr, nbytes, stream)

    def _size(self, n):
        need = int(self._lib.moe_attention_workspace_bytes(n, self.heads, self.head_dim))
        if need == 0:
            raise MoeError(MOE_ERR_INVALID_ARG, "moe_attention_workspace_bytes")
        self._need[n] = need
        return need

    def _out(self, q, qs, out, lse, stream, dev):
        if out is None:
            if stream is not None:  # a tensor made here belongs to the current stream
                raise ValueError("moe: pass out with an explicit stream")
            so = self.heads * self.head_dim
            out = self._empty_like(q) if qs == so else self._empty(q.shape, dtype=self.dtype, device=q.device)
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
        out, so = self._out(q, qs, out, lse, stream, dev)
        if self._many and self._current_device() != dev:  # kernels run on the current device
            self._elsewhere(dev)
        s = self._raw_stream(dev) if stream is None else _stream(stream)
        with self._lock:
            need = _HEADER
            if Tk >= _SPLIT_KEYS:
                if self._sized != (n, Tq, Tk, dev):  # the layers of a model call with the same sizes
                    self._sized_bytes = self._prompt_bytes(n, Tq, Tk, self.heads, self.kv_heads, self.head_dim, self.dt)
                    self._sized = (n, Tq, Tk, dev)
                need = self._sized_bytes
            rec = self._recording(s) if stream is not None or self._capturing() else 0
            ws = None if rec or dev else self._of.get(s)  # the usual case of _Workspaces.get
            if ws is None or ws[1] < need:
                ws = self._ws.get(s, need, dev, rec)
            lse_at = None if lse is None else lse.data_ptr()
            flags = _lib.ATTN_CAUSAL if causal else 0
            ko = None if kv_offsets is None else kv_offsets.data_ptr()
            if len(ws) == 3:
                rc = self._prompt(q.data_ptr(), k.data_ptr(), v.data_ptr(), q_offsets.data_ptr(), ko, n, Tq, Tk,
                                  self.heads, self.kv_heads, self.head_dim, qs, ks, vs, so, self.scale, flags, self.dt,
                                  out.data_ptr(), lse_at, ws[2], ws[1], s)
            else:
                rc = self._prompt_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), q_offsets.data_ptr(), ko, n, Tq, Tk,
                                     self.heads, self.kv_heads, self.head_dim, qs, ks, vs, so, self.scale, flags, self.dt,
                                     out.data_ptr(), lse_at, ws[2], ws[1], ws[3], ws[4], s)
        if rc != MOE_OK:
            raise MoeError(rc, "moe_attention_prompt")
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
        out, so = self._out(q, qs, out, lse, stream, dev)
        if self._many and self._current_device() != dev:  # kernels run on the current device
            self._elsewhere(dev)
        s = self._raw_stream(dev) if stream is None else _stream(stream)
        with self._lock:
            # (the current stream is asked faster than any other)
            rec = self._recording(s) if stream is not None or self._capturing() else 0
            need = self._need.get(n) or self._size(n)
            ws = None if rec or dev else self._of.get(s)  # the usual case of _Workspaces.get
            if ws is None or ws[1] < need:
                ws = self._ws.get(s, need, dev, rec)
            lse_at = None if lse is None else lse.data_ptr()
            if len(ws) == 3:
                rc = self._decode(cache._ref, layer, q.data_ptr(), slots.data_ptr(), n, self.heads, qs, so, shared_len,
                                  self.scale, out.data_ptr(), lse_at, ws[2], ws[1], s)
            else:
                rc = self._decode_ex(cache._ref, layer, q.data_ptr(), slots.data_ptr(), n, self.heads, qs, so,
                                     shared_len, self.scale, out.data_ptr(), lse_at, ws[2], ws[1], ws[3], ws[4], s)
        if rc != MOE_OK:
            raise MoeError(rc, "moe_attention_decode")
        return out
