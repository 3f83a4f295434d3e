"""What the CUDA sources may not hold, by reading them."""

import glob
import os

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_gqa_14_gb300", "csrc")
SOURCES = sorted(f for f in glob.glob(os.path.join(CSRC, "*")) if f.endswith((".cu", ".cuh", ".h", ".c")))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_copy_goes_to_several_ctas(path):
    # The one library serves replicas on several GPUs as well, and does not know whose memory a pool is: every copy
    # is a CTA's own.
    with open(path) as f:
        assert ".multicast::" not in f.read()


def test_the_sources_are_found():
    assert len(SOURCES) > 15
