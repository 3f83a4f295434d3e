"""Refusals that need no GPU: calls that no kernel could run in bounds."""

import pytest
import torch

from paged_kv_gqa_14_gb300 import _lib, ops
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


def test_an_argument_that_is_not_a_number_is_named():
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    pool, s = torch.zeros(1, 16, 1, 64, dtype=torch.int8), torch.ones(1, 1)
    table, one = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    qsl = torch.tensor([0, 1], dtype=torch.int32)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)

    def append(theta=1e6, **kw):
        ops.kv_append_q8(q, q[:, :1], q[:, :1], table, one, qsl, pool, pool, s, s, theta, **kw)

    def attend(scale=0.1, **kw):
        ops.paged_attention_q8(q, pool, pool, s, s, table, one, qsl, scale, out=torch.empty_like(q), workspace=ws, **kw)

    for bad in ("ten", "1.0", None, [1.0]):
        with pytest.raises(TypeError, match="rope_theta must be a number"):
            append(bad)
        with pytest.raises(TypeError, match="scale must be a number"):
            attend(bad)
    for call in (append, attend):
        with pytest.raises(TypeError, match="max_blocks_per_seq must be an integer"):
            call(max_blocks_per_seq=1.0)
    with pytest.raises(TypeError, match="k_cache must be a torch.Tensor"):
        ops.paged_attention_q8(q, None, pool, s, s, table, one, qsl, 0.1, out=torch.empty_like(q), workspace=ws)


def test_fault_injection_kinds(lib):
    for kind in (4, 0):
        assert lib.pkv_set_fault_injection(kind) == 0
    assert lib.pkv_set_fault_injection(5) == 2 and lib.pkv_set_fault_injection(6) == 2
