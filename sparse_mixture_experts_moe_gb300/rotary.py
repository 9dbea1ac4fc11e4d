"""Rotary positions of queries and keys, with a norm of each head in front (moe_rotary_* of include/moe.h).

    rope = Rotary(head_dim=128, base=10000.0)
    q, k = rope.apply(q, positions, k)                                     # turned by their positions
    q, k = rope.apply(q, positions, k, q_weight=wq, k_weight=wk)           # each head normed first, in the same pass
    q = cache.append(k, v, slots, offsets, pos, rope, layer=l, q=q)        # keys turned on their way into the cache

A Rotary is a table of frequencies in host memory: it serves any device, stream and thread. Calls are enqueued on the
current stream, or on `stream`, can be recorded into a graph, and need no workspace.
"""
from __future__ import annotations

import ctypes

from . import _lib
from ._lib import MOE_ERR_INVALID_ARG, MOE_OK, MoeError, _allocator, _stream

_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {None: 0, "linear": 1, "base": 2, "turns": 3, "pairs": 4}


class _Rotary(ctypes.Structure):
    """moe_rotary."""
    _fields_ = [("D", ctypes.c_int), ("R", ctypes.c_int), ("layout", ctypes.c_int), ("magnitude", ctypes.c_float),
                ("turns", ctypes.c_uint64 * 128)]


# The checks below run on every call, where a decode step's kernel takes a few microseconds: each looks at a tensor's
# attributes once and formats a message only when it refuses.
def _tokens(t, name, dim, dtype, dev):
    """Checks a [T, heads, dim] tensor on CUDA device `dev` whose heads are dense within a token; returns (T, heads, token
    stride)."""
    if t.dim() != 3 or t.dtype is not dtype or t.get_device() != dev:
        _not_tokens(t, name, dim, dtype, dev)
    T, n, d = t.shape
    st, sh, sd = t.stride()
    if d != dim or ((sd != 1 or (sh != dim and n > 1)) and T > 0):
        _not_tokens(t, name, dim, dtype, dev)
    return T, n, (st if T > 1 else n * dim)  # (a single token's stride means nothing)


def _not_tokens(t, name, dim, dtype, dev):
    raise ValueError(f"moe: expected {name} [T, heads, {dim}] in {dtype} on cuda:{dev}, heads dense within a token, got "
                     f"{tuple(t.shape)} in {t.dtype} on {t.device} (strides {t.stride()})")


def _result(t, name, T, heads, dim, dtype, dev):
    """Checks an output [T, heads, dim]; returns its token stride."""
    n, h, stride = _tokens(t, name, dim, dtype, dev)
    if n != T or h != heads:
        raise ValueError(f"moe: expected {name} [{T}, {heads}, {dim}], got {tuple(t.shape)}")
    return stride


def _weight(w, name, dim, dtype, dev):
    """Address of a norm's weights."""
    if w.dim() != 1 or w.shape[0] != dim or w.dtype is not dtype or w.get_device() != dev or not w.is_contiguous():
        raise ValueError(f"moe: {name} must be a contiguous [{dim}] tensor in {dtype} on cuda:{dev}")
    return w.data_ptr()


def _apart(a, b):
    """Whether two [T, heads, dim] tensors share no element: their extents do not meet, or they are different heads of one
    fused tensor."""
    size = a.element_size()
    at, bt = a.data_ptr(), b.data_ptr()
    end = [p + ((x.shape[0] - 1) * x.stride()[0] + x.shape[1] * x.shape[2]) * size for p, x in ((at, a), (bt, b))]
    if at >= end[1] or bt >= end[0]:
        return True
    row = a.stride()[0] * size
    if row == 0 or a.stride()[0] != b.stride()[0] or a.shape[0] < 2 or b.shape[0] < 2:  # (0: one row, broadcast)
        return False
    off = (bt - at) % row  # of b's heads behind a's in a token's row
    return off >= a.shape[1] * a.shape[2] * size and off + b.shape[1] * b.shape[2] * size <= row


def _check_overlap(outs, inputs):
    """Refuses outputs that share memory with each other, or with an input that is not the very same tensor: a warp might write
    there before another has read it."""
    outs = [(name, o) for name, o in outs if o is not None]
    for i, (name, o) in enumerate(outs):
        for x, theirs in zip(inputs, ("out", "k_out", "")):
            if x is None:
                continue
            same = (name == theirs or name == "q_out" and theirs == "out") and o.data_ptr() == x.data_ptr() and (
                o.stride()[0] == x.stride()[0] or o.shape[0] < 2)
            if not same and not _apart(o, x):
                raise ValueError(f"moe: {name} overlaps an input without being that input")
        for other, p in outs[i + 1:]:
            if not _apart(o, p):
                raise ValueError(f"moe: {name} and {other} overlap")


class Rotary:
    """Positions as rotations of pairs of a head's first rotary_dim elements (all of them by default): elements p and
    p + rotary_dim / 2 in the "half" layout, 2p and 2p + 1 in the "interleaved" one, by position * base^(-2p / rotary_dim).

    scaling, for contexts longer than the original_len positions trained on: "linear" divides every frequency by `factor`;
    "base" takes base * factor^(rotary_dim / (rotary_dim - 2)); "turns" divides the frequencies of pairs that make at most
    `low` turns over original_len (1 by default), keeps those of at least `high` (4), and goes over linearly in the turns
    between; "pairs" goes over linearly in the pair's number between the pairs of `high` (32) and of `low` (1) turns,
    rounded outwards. magnitude multiplies cosine and sine: 1 by default, 0.1 ln factor + 1 with "pairs".
    frequencies: rotary_dim / 2 numbers in radians a position, in place of all that."""

    def __init__(self, head_dim, rotary_dim=None, base=10000.0, layout="half", scaling=None, factor=1.0, original_len=0,
                 low=None, high=None, magnitude=None, frequencies=None):
        import torch
        if layout not in _LAYOUTS:
            raise ValueError(f"Rotary: layout must be one of {sorted(_LAYOUTS)}, got {layout!r}")
        if scaling not in _SCALINGS:
            raise ValueError(f"Rotary: scaling must be None, 'linear', 'base', 'turns' or 'pairs', got {scaling!r}")
        self._made = (head_dim, rotary_dim, base, layout, scaling, factor, original_len, low, high, magnitude, frequencies)
        self.head_dim = int(head_dim)
        self.rotary_dim = self.head_dim if rotary_dim is None else int(rotary_dim)
        self.layout, self.scaling = layout, scaling
        self._c = _Rotary()
        self._ref = ctypes.addressof(self._c)
        self._lib = _lib.lib()
        if magnitude is not None and not float(magnitude):
            raise ValueError("Rotary: magnitude must not be 0")
        if frequencies is not None:
            if scaling is not None:
                raise ValueError("Rotary: frequencies are taken as they are: scaling must be None")
            f = frequencies = [float(x) for x in frequencies]
            self._made = self._made[:-1] + (f,)
            if len(f) != self.rotary_dim // 2:
                raise ValueError(f"Rotary: expected {self.rotary_dim // 2} frequencies, got {len(f)}")
            f = (ctypes.c_double * max(1, len(f)))(*f)
            rc = self._lib.moe_rotary_set(self._ref, self.head_dim, self.rotary_dim, _LAYOUTS[layout], ctypes.addressof(f),
                                          1.0 if magnitude is None else float(magnitude))
        else:
            low = 1.0 if low is None else float(low)
            high = (4.0 if scaling == "turns" else 32.0) if high is None else float(high)
            rc = self._lib.moe_rotary_init(self._ref, self.head_dim, self.rotary_dim, _LAYOUTS[layout], float(base),
                                           _SCALINGS[scaling], float(factor), int(original_len), low, high,
                                           0.0 if magnitude is None else float(magnitude))
        if rc == MOE_ERR_INVALID_ARG:
            raise ValueError("Rotary: head_dim is a multiple of 8 from 8 to 256, rotary_dim even and at most head_dim, base above 1, "
                             "factor at least 1, 0 < low < high; 'turns' and 'pairs' need original_len, 'base' a rotary_dim other than 2")
        if rc != MOE_OK:
            raise MoeError(rc, "moe_rotary_init")
        self._i32 = torch.int32
        self._dtypes = {torch.bfloat16: _lib.MOE_DTYPE_BF16, torch.float32: _lib.MOE_DTYPE_F32}
        self._new = _allocator(torch)
        self._call = self._lib.moe_rotary_apply
        self._last = self._last_outs = (None, None)
        self._raw_stream = torch._C._cuda_getCurrentRawStream
        self._current_device, self._many = torch._C._cuda_getDevice, torch.cuda.device_count() > 1

    def __reduce__(self):  # copies and pickles are made anew: they have a table of their own
        return Rotary, self._made

    @property
    def magnitude(self):
        return float(self._c.magnitude)

    @property
    def frequencies(self):
        """The pairs' frequencies, radians a position (below a whole turn)."""
        return [self._c.turns[p] * 2.0 ** -64 * 6.283185307179586 for p in range(self.rotary_dim // 2)]

    def apply(self, q, positions, k=None, q_weight=None, k_weight=None, eps=1e-6, out=None, k_out=None, stream=None):
        """q [T, heads, head_dim] and k [T, kv_heads, head_dim] (optional) of the tokens at positions [T] (int32, any sign).
        With q_weight / k_weight [head_dim] (their type) each head is first x / sqrt(mean x^2 + eps) * weight. Returns q's
        result, or (q's, k's) where there is k; out and k_out may be q and k themselves."""
        # What the tensors look like decides everything but their addresses: a call like the last one is not checked again.
        look = (q.shape, q.stride(), q.dtype, q.get_device(), positions.shape, positions.dtype, positions.get_device(),
                positions.is_contiguous(),
                k if k is None else (k.shape, k.stride(), k.dtype, k.get_device()),
                q_weight if q_weight is None else (q_weight.shape, q_weight.dtype, q_weight.get_device(), q_weight.is_contiguous()),
                k_weight if k_weight is None else (k_weight.shape, k_weight.dtype, k_weight.get_device(), k_weight.is_contiguous()))
        last = self._last
        if last[0] != look:
            last = self._last = (look, self._checked(q, positions, k, q_weight, k_weight))
        dev, dtype, dt, T, H, qs, Hk, ks, q_new, k_new = last[1]
        if self._many and self._current_device() != dev:  # kernels run on the current device
            raise ValueError(f"moe: the tensors are on cuda:{dev}, which is not the current device (torch.cuda.device)")
        if out is None and k_out is None:
            if stream is not None:  # tensors made here belong to the current stream
                raise ValueError("moe: pass out (and k_out) with an explicit stream")
            out, qso = self._new(*q_new), H * self.head_dim
            if k is not None:
                k_out = self._new(*k_new)
            kso = Hk * self.head_dim
        else:
            out, qso, k_out, kso = self._outs(q, k, out, k_out, last[1], stream)
        rc = self._call(self._ref, q.data_ptr(), qs, H, k if k is None else k.data_ptr(), ks, Hk, positions.data_ptr(), T, dt,
                        q_weight if q_weight is None else q_weight.data_ptr(), k_weight if k_weight is None else k_weight.data_ptr(),
                        eps, out.data_ptr(), qso, k if k is None else k_out.data_ptr(), kso,
                        self._raw_stream(dev) if stream is None else _stream(stream))
        if rc != MOE_OK:
            raise MoeError(rc, "moe_rotary_apply")
        return out if k is None else (out, k_out)

    def _checked(self, q, positions, k, q_weight, k_weight):
        dev, dtype, D = q.get_device(), q.dtype, self.head_dim
        if dev < 0:
            raise ValueError(f"moe: q must be a CUDA tensor (got one on {q.device})")
        dt = self._dtypes.get(dtype)
        if dt is None:
            raise TypeError(f"unsupported dtype {dtype}")
        T, H, qs = _tokens(q, "q", D, dtype, dev)
        if H == 0:
            raise ValueError("moe: q has no heads")
        if (positions.dtype is not self._i32 or positions.get_device() != dev or positions.shape != (T,)
                or not positions.is_contiguous()):
            raise ValueError(f"moe: positions must be a contiguous int32 tensor [{T}] on cuda:{dev}")
        for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            if w is not None:
                _weight(w, name, D, dtype, dev)
        if k is None:
            if k_weight is not None:
                raise ValueError("moe: k_weight needs k")
            Hk = ks = 0
        else:
            Tk, Hk, ks = _tokens(k, "k", D, dtype, dev)
            if Tk != T or Hk == 0:
                raise ValueError(f"moe: q has {T} tokens, k {Tk} with {Hk} heads")
        return dev, dtype, dt, T, H, qs, Hk, ks, ((T, H, D), (H * D, D, 1), dtype), ((T, Hk, D), (Hk * D, D, 1), dtype)

    def _outs(self, q, k, out, k_out, call, stream):
        """Outputs of which the caller gave one or both, and their token strides."""
        dev, dtype, _, T, H, qs, Hk, ks, q_new, k_new = call
        if stream is not None and (out is None or (k is not None and k_out is None)):
            raise ValueError("moe: pass out (and k_out) with an explicit stream")
        if k is None and k_out is not None:
            raise ValueError("moe: k_out needs k")
        if out is None:
            out = self._new(*q_new)
        if k is not None and k_out is None:
            k_out = self._new(*k_new)
        look = (call, out.shape, out.stride(), out.dtype, out.get_device(),
                k if k is None else (k_out.shape, k_out.stride(), k_out.dtype, k_out.get_device()))
        last = self._last_outs
        if last[0] != look:
            qso, kso, D = _result(out, "out", T, H, self.head_dim, dtype, dev), 0, self.head_dim
            if k is not None:
                kso = _result(k_out, "k_out", T, Hk, D, dtype, dev)
            size = q.element_size()  # and the bytes from the first element's to the last's end
            ends = [((T - 1) * s + h * D) * size if h else 0 for s, h in ((qso, H), (kso, Hk), (qs, H), (ks, Hk))]
            last = self._last_outs = (look, (qso, kso, *ends))
        qso, kso, n_out, n_k_out, n_q, n_k = last[1]
        if T > 0:
            o, x = out.data_ptr(), q.data_ptr()
            fine = o + n_out <= x or x + n_q <= o or (o == x and qso == qs)
            if k is not None:
                p, y = k_out.data_ptr(), k.data_ptr()
                fine = (fine and (p + n_k_out <= y or y + n_k <= p or (p == y and kso == ks)) and (o + n_out <= p or p + n_k_out <= o)
                        and (o + n_out <= y or y + n_k <= o) and (p + n_k_out <= x or x + n_q <= p))
            if not fine:  # (heads of one fused tensor lie between each other)
                _check_overlap((("out", out), ("k_out", k_out)), (q, k))
        return out, qso, k_out, kso
