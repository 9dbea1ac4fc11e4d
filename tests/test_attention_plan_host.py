"""A cache's plan holds for that cache alone. Needs no GPU: an fp32 cache's plan holds no descriptors."""
import ctypes

import sparse_mixture_experts_moe_gb300 as moe
from sparse_mixture_experts_moe_gb300 import _lib
from test_attention_host import cache, decode


def planned(**kw):
    c = cache(**kw)
    n = _lib.lib().moe_cache_plan_bytes()
    buf = ctypes.create_string_buffer(n)
    assert _lib.lib().moe_cache_plan(ctypes.addressof(c), ctypes.addressof(buf), n) == moe.MOE_OK
    c.plan = ctypes.addressof(buf)
    return c, buf


def test_a_plan_of_another_type_is_refused():
    """The plan of an fp32 cache holds empty descriptors: the same arrays as bf16 must not be copied by them."""
    c, _keep = planned(dt=moe.MOE_DTYPE_F32)
    c.dt = moe.MOE_DTYPE_BF16
    assert decode(c) == moe.MOE_ERR_INVALID_ARG
    assert decode(c, shared=0) == moe.MOE_ERR_INVALID_ARG


def test_a_plan_is_checked_where_no_descriptors_are_used():
    """fp32 caches and heads of more than 128 take no descriptors; a plan of another cache is refused there too."""
    c, _keep = planned(dt=moe.MOE_DTYPE_F32)
    for name, value in (("n_pages", 101), ("n_layers", 1), ("page_size", 32)):
        other = cache(dt=moe.MOE_DTYPE_F32, **{name: value})
        other.plan = c.plan
        assert decode(other) == moe.MOE_ERR_INVALID_ARG
    wide = cache(D=256)
    wide.plan = c.plan
    lib = _lib.lib()
    assert decode(wide, qs=2048, os=2048, bytes=lib.moe_attention_workspace_bytes(3, 8, 256)) == moe.MOE_ERR_INVALID_ARG
