"""Refusals that need no GPU: calls that no kernel could run in bounds."""

import pytest

from paged_kv_gqa_14_gb300 import _lib
from paged_kv_gqa_14_gb300 import build as B
from tests.test_abi import _attn as attn
from tests.test_q8 import _attn as attn_q8


@pytest.fixture(scope="module")
def lib():
    B.build()
    return _lib.load()


def test_attention_refuses_a_pool_of_no_blocks(lib):
    # a block id outside the pool is read as block 0, which there is not
    for call in (attn, attn_q8):
        assert call(lib, nb=0) == 2
        assert call(lib, nb=0, T=0) == 0 and call(lib, nb=0, B=0) == 0
