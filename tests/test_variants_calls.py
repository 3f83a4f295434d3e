"""Calls of the attention variants that their documentation does not allow, without a GPU."""

import pytest

from paged_kv_gqa_14_gb300 import build as B
from paged_kv_gqa_14_gb300 import ops


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


@pytest.mark.parametrize("sizes", [(2**32 + 32, 128), (32, 2**32 + 128), (-(2**32) + 32, 128), (32, 2**31)])
def test_bucket_sizes_past_32_bits_are_refused(sizes):
    with pytest.raises(ValueError, match="must fit 32 bits"):
        ops.relative_buckets(*sizes)


@pytest.mark.parametrize("kw", [dict(num_buckets=32.5, max_distance=128), dict(num_buckets=32, max_distance=127.5),
                                dict(starts=[0, 1.5]), dict(starts=["0", "3"])])
def test_buckets_of_no_whole_numbers_are_refused(kw):
    with pytest.raises(ValueError, match="whole numbers"):
        ops.relative_buckets(**kw)


def test_whole_numbers_of_any_kind_are_taken():
    want = list(ops.relative_buckets(32, 128).starts)
    assert list(ops.relative_buckets(32.0, 128.0).starts) == want
    assert list(ops.relative_buckets(starts=[float(x) for x in want[:32]]).starts) == want
