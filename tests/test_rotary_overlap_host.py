"""Which outputs share memory with what a call reads. Needs no GPU: addresses and strides alone count."""
import pytest
import torch

from sparse_mixture_experts_moe_gb300.rotary import _apart, _check_overlap


def test_heads_of_one_fused_tensor_are_apart():
    x = torch.zeros(4, 6, 8)
    assert _apart(x[:, :2], x[:, 2:4]) and _apart(x[:, 4:], x[:, :4]) and _apart(x[1:3, :2], x[:2, 2:])
    assert not _apart(x[:, :3], x[:, 2:4]) and not _apart(x[:2, :2], x[1:, :2])


def test_broadcast_tensors_overlap():
    """One token's row for all tokens (stride 0)."""
    x = torch.zeros(1, 6, 8)
    q, k = x[:, :2].expand(4, 2, 8), x[:, 2:4].expand(4, 2, 8)
    assert not _apart(q, q) and _apart(q, k)
    with pytest.raises(ValueError, match="overlaps an input"):
        _check_overlap((("k_out", q),), (q, None))
