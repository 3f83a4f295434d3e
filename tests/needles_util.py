"""Weights of single keys, read out of an attention: V is zero but for one 1 in a column for each of as many keys as an
output row has columns, so that a column of the output is the weight of its key.  A key that is lost, or counted twice, is
off by all of its weight, however many others there are.

The bound: a weight is rounded (or cut) to bf16 and divided by the sum of the rounded ones, and the output rounded, each
within 2^-8 of its value (a cut one lies in (-2^-7, 0], which its quotient with a sum of cut ones turns into 2^-7 either way, as
two roundings do); a score's error e, to first order, is 2 e of the quotient, as in ``oracle.variants``.  So a column of one
map is off by at most 1.02 (3 x 2^-8 + 4 e + 2^-15) of its weight, and one of a difference by that of its two weights' sum."""

import numpy as np

from oracle import attention as OA
from oracle import variants as OV
from oracle.bf16 import bf16_bits_to_f64


def weights(Q, K, scale, first, bias=None):
    """(softmax weights [n, ctx], error of a score [n]) of rows at positions first .. first + n - 1."""
    n, ctx = Q.shape[0], K.shape[0]
    s, size = scale * (Q @ K.T), scale * (np.abs(Q) @ np.abs(K).T)
    if bias is not None:
        s, size = s + bias, size + np.abs(bias) * 2.0**-6
    seen = np.arange(ctx)[None, :] <= first + np.arange(n)[:, None]
    s = np.where(seen, s, -np.inf)
    w = np.exp(s - s.max(axis=1, keepdims=True))
    return w / w.sum(axis=1, keepdims=True), OV.SUM_FP32 * np.where(seen, size, 0.0).max(axis=1)


def rel_bound(e):
    return 1.02 * (3 * OV.HALF_BF16 + 4 * e + 2.0**-15)


def keys_of(batch):
    """K of each sequence [ctx, hkv, d] (V is not looked at)."""
    b = batch.bt
    zero = np.zeros_like(batch.kc)
    return [OA.gather_sequence_kv(batch.kc, zero, b.block_tables[i], int(n))[0] for i, n in enumerate(b.context_lens)]


def spans_of(batch):
    """(sequence, its first row, rows, position of its first row)"""
    b = batch.bt
    for i, n in enumerate(b.context_lens):
        s0, s1 = int(b.query_start_loc[i]), int(b.query_start_loc[i + 1])
        if s1 > s0:
            yield i, s0, s1 - s0, int(n) - (s1 - s0)


def bias_weights(batch, bias, starts):
    """For each span and q head the weights and their relative bound: [(rows, head, w [n, ctx], bound [n, ctx])]."""
    K, G, out = keys_of(batch), batch.hq // batch.hkv, []
    bucket = np.array([OV.bucket_of(x, starts) for x in range(int(starts[-1]) + 1)])
    for i, s0, n, first in spans_of(batch):
        Q = bf16_bits_to_f64(batch.q[s0:s0 + n])
        back = np.clip(first + np.arange(n)[:, None] - np.arange(first + n)[None, :], 0, len(bucket) - 1)
        for h in range(batch.hq):
            w, e = weights(Q[:, h], K[i][:, h // G], batch.scale, first, bias[:, h][bucket[back]])
            out.append((i, slice(s0, s0 + n), h, w, rel_bound(e)[:, None] * w))
    return out


def diff_weights(batch, lam):
    """The same for each head of a difference: a_0 - lam a_1."""
    K, G, out = keys_of(batch), batch.hq // batch.hkv, []
    for i, s0, n, first in spans_of(batch):
        Q = bf16_bits_to_f64(batch.q[s0:s0 + n])
        for h in range(batch.hq // 2):
            g = h // G
            (w0, e0), (w1, e1) = (weights(Q[:, 2 * h + c], K[i][:, 2 * g + c], batch.scale, first) for c in (0, 1))
            out.append((i, slice(s0, s0 + n), h, w0 - lam * w1,
                        rel_bound(np.maximum(e0, e1))[:, None] * (w0 + abs(lam) * w1)))
    return out


def off(got, want, bound):
    """How many of a call's columns are past their bound (a weight below 2^-120 may be nothing)."""
    return int(np.count_nonzero(np.abs(got - want) > bound + 2.0**-120))
