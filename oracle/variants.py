"""Attention with a bucketed relative position bias, and differential attention, over the paged cache in fp64 (test
infrastructure only).

Rows, spans and masks as in ``attention.py``.  Beside the outputs each function returns how far an output of the
given roundings may be off to first order; the derivation stands at ``slack_of_map``.
"""

import numpy as np

from .attention import gather_sequence_kv
from .bf16 import bf16_bits_to_f64

HALF_BF16 = 2.0**-8  # half a step of bf16, relative to the value
SUM_FP32 = 2.0**-16  # 128 products summed in fp32 with up to 2^-23 of the sum of magnitudes lost at each


def bucket_of(n, starts):
    """The last i with starts[i] <= n, by looking at each."""
    i = 0
    for j, s in enumerate(starts):
        if s <= n:
            i = j
    return i


def log_starts(num_buckets, max_distance):
    """The usual buckets' least distances, from the formula's floor by whole numbers."""
    e = num_buckets // 2
    k = num_buckets - e
    starts = list(range(e))
    for j in range(k):
        n = e
        while n**k < max_distance**j * e ** (k - j):
            n += 1
        starts.append(n)
    return starts


def _map(Q, K, V, scale, first, bias=None):
    """One softmax map applied to V: rows at positions first .. first + n - 1; bias [n, ctx] or None.
    Returns (o [n, W], spread [n, W] = sum_j w_j |v_j - o|, error of a score [n])."""
    n, ctx = Q.shape[0], K.shape[0]
    S = scale * (Q @ K.T)
    size = np.abs(scale) * (np.abs(Q) @ np.abs(K).T)
    if bias is not None:
        S = S + bias
        # (its sum with the score and with log2(e) rounded in fp32; one that swallows every score in 64 bits as well
        # leaves no error between the keys that share it)
        size = size + np.where(np.abs(bias) < 1e20, np.abs(bias), 0.0) * 2.0**-6
    seen = np.arange(ctx)[None, :] <= first + np.arange(n)[:, None]
    S = np.where(seen, S, -np.inf)
    size = np.where(seen & np.isfinite(S), size, 0.0).max(axis=1)
    m = S.max(axis=1, keepdims=True)
    w = np.exp(S - np.where(np.isfinite(m), m, 0.0))
    total = w.sum(axis=1, keepdims=True)
    w = w / np.where(total == 0, 1.0, total)  # a row without keys: zeros
    o = w @ V
    # sum_j w_j |v_j - o| <= sqrt(sum_j w_j (v_j - o)^2), the weights being a distribution
    var = np.maximum(w @ (V * V) - o * o, 0.0)
    return o, np.sqrt(var), SUM_FP32 * size


def slack_of_map(spread, score_error, weight_error=HALF_BF16):
    """How far one map's output may be off: each weight is rounded to bf16 and divided by the sum of the rounded
    ones, and its score has an error e, so weight j changes by a factor 1 + d_j with |d_j| <= 2^-8 + 2 e + 2^-16 (the
    power's own error, and l's and O's sums) and the output by sum_j w_j d_j (v_j - o) to first order, at most
    max|d| sum_j w_j |v_j - o|.  Weights that are cut to bf16 instead change by -2^-7 < d_j <= 0: since sum_j w_j (v_j - o)
    = 0, d_j may be taken 2^-8 higher throughout, and the bound is the same.  (A factor 1.02 for the second order.)  Weights kept in
    more bits have a ``weight_error`` of their own."""
    return 1.02 * (weight_error + 2.0 * score_error[:, None] + 2.0**-16) * spread


def paged_attention_bias(q, k_cache, v_cache, block_tables, context_lens, query_start_loc, scale, bias, starts):
    """Returns (out [T, Hq, d], slack), NaN in rows that no span covers; bias [num_buckets, Hq] as float64."""
    T, Hq, d = q.shape
    G = Hq // k_cache.shape[2]
    out, slack = np.full((T, Hq, d), np.nan), np.full((T, Hq, d), np.nan)
    for b, ctx in enumerate(np.asarray(context_lens).astype(np.int64)):
        s0, s1 = int(query_start_loc[b]), int(query_start_loc[b + 1])
        n = s1 - s0
        if n == 0:
            continue
        K, V = gather_sequence_kv(k_cache, v_cache, block_tables[b], ctx)
        Q = bf16_bits_to_f64(q[s0:s1])
        first = int(ctx) - n
        far = int(starts[-1])
        table = np.array([bucket_of(x, starts) for x in range(min(int(ctx), far + 1))])
        back = np.clip(first + np.arange(n)[:, None] - np.arange(int(ctx))[None, :], 0, len(table) - 1)
        for h in range(Hq):
            o, spread, e = _map(Q[:, h], K[:, h // G], V[:, h // G], scale, first, bias[:, h][table[back]])
            out[s0:s1, h] = o
            slack[s0:s1, h] = HALF_BF16 * np.abs(o) + slack_of_map(spread, e) + 2.0**-20 * np.abs(o)
    return out, slack


def paged_attention_diff(q, k_cache, v_cache, block_tables, context_lens, query_start_loc, scale, lam,
                         norm_weight=None, norm_eps=1e-5, out_scale=1.0, weight_error=HALF_BF16):
    """Returns (out [T, Hq / 2, 2 d], slack); lam [Hq / 2] or [T, Hq / 2]; ``weight_error`` as for ``slack_of_map``."""
    T, Hq, d = q.shape
    G = Hq // k_cache.shape[2]
    H = Hq // 2
    lam = np.broadcast_to(np.asarray(lam, dtype=np.float64), (T, H))
    out, slack = np.full((T, H, 2 * d), np.nan), np.full((T, H, 2 * d), np.nan)
    for b, ctx in enumerate(np.asarray(context_lens).astype(np.int64)):
        s0, s1 = int(query_start_loc[b]), int(query_start_loc[b + 1])
        n = s1 - s0
        if n == 0:
            continue
        K, V = gather_sequence_kv(k_cache, v_cache, block_tables[b], ctx)
        Q = bf16_bits_to_f64(q[s0:s1])
        first = int(ctx) - n
        for h in range(H):
            g = h // G
            both = np.concatenate([V[:, 2 * g], V[:, 2 * g + 1]], axis=1)
            o0, sp0, e0 = _map(Q[:, 2 * h], K[:, 2 * g], both, scale, first)
            o1, sp1, e1 = _map(Q[:, 2 * h + 1], K[:, 2 * g + 1], both, scale, first)
            la = lam[s0:s1, h, None]
            x = o0 - la * o1
            # the maps' errors, and the subtraction's in fp32
            dx = slack_of_map(sp0, e0, weight_error) + np.abs(la) * slack_of_map(sp1, e1, weight_error)
            dx = dx + 2.0**-20 * (np.abs(o0) + np.abs(la * o1))
            if norm_weight is None:
                y, dy = x, dx
            else:
                # y = w x / r, r = sqrt(mean x^2 + eps): dr <= sqrt(mean dx^2), dy <= |w| (dx + |x| dr / r) / (r - dr)
                r = np.sqrt((x * x).mean(axis=1, keepdims=True) + norm_eps)
                dr = np.sqrt((dx * dx).mean(axis=1, keepdims=True))
                w = np.asarray(norm_weight, dtype=np.float64)[None, :]
                y = w * x / r
                dy = np.where(dr < r, np.abs(w) * (dx + np.abs(x) * dr / r) / np.maximum(r - dr, 1e-300), np.inf)
            out[s0:s1, h] = out_scale * y
            slack[s0:s1, h] = np.abs(out_scale) * (dy + (HALF_BF16 + 2.0**-18) * (np.abs(y) + dy))
    return out, slack
