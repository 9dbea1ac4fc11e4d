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
from ._lib import MOE_ERR_INVALID_ARG, MOE_OK, MoeError, _stream

_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {None: 0, "linear": 1, "base": 2, "turns": 3, "pairs": 4}


class _Rotary(ctypes.Structure):
    """moe_rotary."""
    _fields_ = [("D", ctypes.c_int), ("R", ctypes.c_int), ("layout", ctypes.c_int), ("magnitude", ctypes.c_float),
                ("turns", ctypes.c_uint64 * 128)]


def _tokens(t, name, dim, dtype, dev, heads=None):
    """Checks a [T, heads, dim] tensor on CUDA device `dev` whose heads are dense within a token; returns (T, heads, token
    stride)."""
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim or (heads is not None and shape[1] != heads) or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"moe: expected {name} [T, {'heads' if heads is None else heads}, {dim}] in {dtype} on cuda:{dev}, got "
                         f"{tuple(shape)} in {t.dtype} on {t.device}")
    st, sh, sd = t.stride()
    T, n = shape[0], shape[1]
    if T > 0 and (sd != 1 or (sh != dim and n > 1)):
        raise ValueError(f"moe: {name} must have dense heads within a token (strides {t.stride()})")
    return T, n, (st if T > 1 else n * dim)  # (a single token's stride means nothing)


def _weight(w, name, dim, dtype, dev):
    """Address of a norm's weights, None without."""
    if w is None:
        return None
    if w.dim() != 1 or w.shape[0] != dim or w.dtype is not dtype or w.get_device() != dev or not w.is_contiguous():
        raise ValueError(f"moe: {name} must be a contiguous [{dim}] tensor in {dtype} on cuda:{dev}")
    return w.data_ptr()


def _alone(out, x, name):
    """Refuses an output that shares memory with an input which is not the very same tensor: a warp may write there before
    another has read it."""
    a, b = out.data_ptr(), x.data_ptr()
    if a == b and (out.stride(0) == x.stride(0) or x.shape[0] < 2):
        return
    end_a = a + ((out.shape[0] - 1) * out.stride(0) + out.shape[1] * out.shape[2]) * out.element_size()
    end_b = b + ((x.shape[0] - 1) * x.stride(0) + x.shape[1] * x.shape[2]) * x.element_size()
    if a >= end_b or b >= end_a:
        return
    # slices of one fused tensor: the same token stride, and apart within a token
    row, size = x.stride(0) * x.element_size(), out.element_size() * out.shape[2]
    off = (a - b) % row if out.stride(0) == x.stride(0) else 0
    if not (out.stride(0) == x.stride(0) and off >= x.shape[1] * size and off + out.shape[1] * size <= row):
        raise ValueError(f"moe: {name} overlaps an input without being that input")


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
            f = [float(x) for x in frequencies]
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
        self._empty = torch.empty
        self._raw_stream = torch._C._cuda_getCurrentRawStream
        self._current_device, self._many = torch._C._cuda_getDevice, torch.cuda.device_count() > 1

    @property
    def magnitude(self):
        return float(self._c.magnitude)

    @property
    def frequencies(self):
        """The pairs' frequencies, radians a position (below a whole turn)."""
        return [self._c.turns[p] * 2.0 ** -64 * 6.283185307179586 for p in range(self.rotary_dim // 2)]

    def _out(self, x, out, n, name, T, dtype, dev, stream):
        if out is None:
            if stream is not None:  # a tensor made here belongs to the current stream
                raise ValueError(f"moe: pass {name} with an explicit stream")
            return self._empty((T, n, self.head_dim), dtype=dtype, device=x.device), n * self.head_dim
        to, _, so = _tokens(out, name, self.head_dim, dtype, dev, n)
        if to != T:
            raise ValueError(f"moe: expected {name} {tuple(x.shape)}, got {tuple(out.shape)}")
        return out, so

    def apply(self, q, positions, k=None, q_weight=None, k_weight=None, eps=1e-6, out=None, k_out=None, stream=None):
        """q [T, heads, head_dim] and k [T, kv_heads, head_dim] (optional) of the tokens at positions [T] (int32, any sign).
        With q_weight / k_weight [head_dim] (their type) each head is first x / sqrt(mean x^2 + eps) * weight. Returns q's
        result, or (q's, k's) where there is k; out and k_out may be q and k themselves."""
        dev = q.get_device()
        if dev < 0:
            raise ValueError(f"moe: q must be a CUDA tensor (got one on {q.device})")
        dtype = q.dtype
        dt = self._dtypes.get(dtype)
        if dt is None:
            raise TypeError(f"unsupported dtype {dtype}")
        T, H, qs = _tokens(q, "q", self.head_dim, dtype, dev)
        if positions.dtype is not self._i32 or positions.get_device() != dev or positions.shape != (T,) or not positions.is_contiguous():
            raise ValueError(f"moe: positions must be a contiguous int32 tensor [{T}] on cuda:{dev}")
        wq, wk = _weight(q_weight, "q_weight", self.head_dim, dtype, dev), _weight(k_weight, "k_weight", self.head_dim, dtype, dev)
        if H == 0:
            raise ValueError("moe: q has no heads")
        given, k_given = out, k_out
        if k is None:
            if k_out is not None or k_weight is not None:
                raise ValueError("moe: k_out and k_weight need k")
            Hk, ks, kso, k_at, ko_at = 0, 0, 0, None, None
        else:
            Tk, Hk, ks = _tokens(k, "k", self.head_dim, dtype, dev)
            if Tk != T or Hk == 0:
                raise ValueError(f"moe: q has {T} tokens, k {Tk} with {Hk} heads")
            k_out, kso = self._out(k, k_out, Hk, "k_out", T, dtype, dev, stream)
            k_at, ko_at = k.data_ptr(), k_out.data_ptr()
        out, qso = self._out(q, out, H, "out", T, dtype, dev, stream)
        if T > 0:
            for o, name in ((given, "out"), (k_given, "k_out")):
                if o is not None:
                    for x in (q, k):
                        if x is not None:
                            _alone(o, x, name)
            if given is not None and k_given is not None:
                _alone(given, k_given, "out")
                if given.data_ptr() == k_given.data_ptr():
                    raise ValueError("moe: out and k_out are the same memory")
        if self._many and self._current_device() != dev:  # kernels run on the current device
            raise ValueError(f"moe: the tensors are on cuda:{dev}, which is not the current device (torch.cuda.device)")
        s = self._raw_stream(dev) if stream is None else _stream(stream)
        rc = self._lib.moe_rotary_apply(self._ref, q.data_ptr(), qs, H, k_at, ks, Hk, positions.data_ptr(), T, dt, wq, wk,
                                        float(eps), out.data_ptr(), qso, ko_at, kso, s)
        if rc != MOE_OK:
            raise MoeError(rc, "moe_rotary_apply")
        return out if k is None else (out, k_out)
