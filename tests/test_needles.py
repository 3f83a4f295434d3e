"""The check of single keys' weights (needles_util.py) on the CPU: it passes outputs of the roundings that a call may make and
fails where one key, one page or one tile is lost or counted twice, at the lengths that the GPU's tests use."""

import numpy as np
import pytest
import torch

from tests import needles_util as N


def _bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).double().numpy()


def _cut(x):
    bits = np.ascontiguousarray(x.astype(np.float32)).view(np.uint32) & np.uint32(0xFFFF0000)
    return bits.view(np.float32).astype(np.float64)


def _rows(ctx, d, seed):
    rng = np.random.default_rng(seed)
    return _bf16(rng.normal(size=(3, d))), _bf16(rng.normal(size=(ctx, d)))


def _output(Q, K, scale, first, rounded, times):
    """What a call would give for the needles of every key, ``times`` each key's count (1 unless it is lost or doubled)."""
    n, ctx = Q.shape[0], K.shape[0]
    s = scale * (Q @ K.T)
    s = np.where(np.arange(ctx)[None, :] <= first + np.arange(n)[:, None], s, -np.inf)
    w = rounded(np.exp(s - s.max(axis=1, keepdims=True))) * times
    return _bf16(w / w.sum(axis=1, keepdims=True))


@pytest.mark.parametrize("ctx", (300, 3000, 9000))
@pytest.mark.parametrize("rounded", (_bf16, _cut), ids=("rounded", "cut"))
def test_roundings_pass_and_lost_or_doubled_keys_do_not(ctx, rounded):
    Q, K = _rows(ctx, 128, ctx)
    scale, first = 128**-0.5, ctx - 3
    w, e = N.weights(Q, K, scale, first)
    bound = N.rel_bound(e)[:, None] * w
    ones = np.ones(ctx)
    assert N.off(_output(Q, K, scale, first, rounded, ones), w, bound) == 0
    for count in (0.0, 2.0):
        for at in (slice(0, 1), slice(ctx // 2, ctx // 2 + 1), slice(ctx - 3, ctx - 2), slice(160, 176), slice(128, 256)):
            times = ones.copy()
            times[at] = count
            assert N.off(_output(Q, K, scale, first, rounded, times), w, bound) >= 3 * (at.stop - at.start), (count, at)


def test_weights_are_the_oracle_s():
    Q, K = _rows(40, 64, 1)
    w, _ = N.weights(Q, K, 0.125, 37)
    V = np.random.default_rng(2).normal(size=(40, 64))
    for r in range(3):
        s = np.exp(0.125 * (Q[r] @ K[: 38 + r].T))
        np.testing.assert_allclose(w[r] @ V, (s / s.sum()) @ V[: 38 + r], rtol=1e-12, atol=1e-14)
