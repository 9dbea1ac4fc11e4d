"""Sizes at the end of 32 bits, where a block of keys would end past them."""
import pytest

import sparse_mixture_experts_moe_gb300 as moe
from test_attention_host import FAKE, cache, decode, prompt

MOST = 2 ** 31 - 256


@pytest.mark.parametrize("keys", [2 ** 31 - 1, 2 ** 31 - 128, MOST + 1])
def test_prompts_over_too_many_keys_are_refused(keys):
    assert prompt(Tq=1, n=1, Tkv=keys, ko=FAKE, qs=512) == moe.MOE_ERR_INVALID_ARG
    assert prompt(Tq=1, n=1, Tkv=keys, ko=FAKE, dt=0) == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("page", [16, 64, 256])
def test_caches_of_too_long_sequences_are_refused(page):
    for width in (MOST // page + 1, (2 ** 31 - 1) // page):
        if width * page <= MOST:
            continue
        c = cache(table_width=width, page_size=page, n_slots=1)
        assert decode(c, n=0) == moe.MOE_ERR_INVALID_ARG
    assert decode(cache(table_width=MOST // page, page_size=page, n_slots=1), n=0, shared=0) == moe.MOE_OK
