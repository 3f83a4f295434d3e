"""Every key's weight in the attention variants, one by one (needles_util.py): pieces, pages, tiles and shared ranges lose
none and count none twice, however many keys there are."""

import numpy as np
import pytest
import torch

from oracle import variants as OV
from paged_kv_gqa_14_gb300 import ops
from tests import needles_util as N
from tests import variants_util as U

pytestmark = pytest.mark.gpu

T5 = (32, 128)


def _each_key(batch, per, call, columns_of, expected, what):
    """``call(v)`` for V with needles at ``per`` keys of every sequence at a time, against ``expected``."""
    _, _, vc, bt, ctx, _, _ = batch.dev()
    bs = vc.shape[1]
    empty = torch.where(vc.isnan(), vc, torch.zeros_like(vc))
    table, lens = bt.long().cpu(), ctx.cpu()
    for start in range(0, int(lens.max()), per):
        v = empty.clone()
        for i, n in enumerate(lens.tolist()):
            if start < n:
                keys = torch.arange(start, min(start + per, n))
                columns_of(v, table[i, keys // bs].cuda(), (keys % bs).cuda(), torch.arange(len(keys)).cuda())
        got = call(v).double().cpu().numpy()
        for i, rows, h, w, bound in expected:
            m = min(per, w.shape[1] - start)
            if m > 0:
                part = slice(start, start + m)
                bad = N.off(got[rows, h, :m], w[:, part], bound[:, part])
                assert bad == 0, f"{what}: sequence {i} head {h} keys {start} .. {start + m - 1}: {bad} off"
    assert ops.get_device_error() == 0


def each_key_of_the_bias(batch, seed=0, **kw):
    q, kc, _, bt, ctx, qsl, scale = batch.dev()
    bias, bias64 = U.bias_of(batch, T5[0], seed)
    bias, buckets = bias.cuda(), ops.relative_buckets(*T5)

    def one_hot(v, block, slot, column):
        v[block, slot, :, column] = 1.0

    _each_key(batch, batch.d, lambda v: ops.paged_attention_bias(q, kc, v, bt, ctx, qsl, scale, bias, buckets, **kw), one_hot,
              N.bias_weights(batch, bias64, OV.log_starts(*T5)), "bias")


def each_key_of_the_difference(batch, lam=-0.5, **kw):
    """lam below 0: no weight of one map hides behind the other's."""
    q, kc, _, bt, ctx, qsl, scale = batch.dev()
    lams, d = torch.full((batch.hq // 2,), lam, device="cuda"), batch.d

    def one_hot(v, block, slot, column):
        for part in (0, 1):  # the pair's two v heads are an output row's two halves
            here = (column // d) == part
            for head in range(part, batch.hkv, 2):
                v[block[here], slot[here], head, column[here] - part * d] = 1.0

    _each_key(batch, 2 * d, lambda v: ops.paged_attention_diff(q, kc, v, bt, ctx, qsl, scale, lams, **kw), one_hot,
              N.diff_weights(batch, lam), "difference")


CASES = {
    # decode: entries in pieces, whole, many to a CTA; both page layouts
    "9000 keys": dict(ctx=[9000], spans=[1], hq=8, hkv=4, d=128, bs=64),
    "two long, one short": dict(ctx=[5003, 1, 4097], spans=[1, 1, 1], hq=4, hkv=2, d=64),
    "blocks of 8": dict(ctx=[2049, 777, 16], spans=[1, 1, 1], hq=16, hkv=8, d=128, bs=8),
    "joined in the decode": dict(ctx=[900, 64, 513, 130], spans=[1] * 4, hq=8, hkv=2, d=64),
    "a span among decode rows": dict(ctx=[900, 5, 6, 7, 30], spans=[4, 0, 0, 0, 1], hq=8, hkv=4, d=128),
    # prefill: whole items, many of them, items shared by pairs of CTAs, ends inside tiles
    "a chunk": dict(ctx=[3300], spans=[300], hq=4, hkv=2, d=128, bs=32),
    "a prompt": dict(ctx=[1500], spans=[1500], hq=2, hkv=2, d=64),
    "many items": dict(ctx=[700, 411, 129, 530] * 4, spans=[60, 38, 33, 130] * 4, hq=16, hkv=8, d=64),
    "shared": dict(ctx=[3000], spans=[12], hq=12, hkv=4, d=128),
    "shared, some not": dict(ctx=[2000, 700, 40], spans=[9, 2, 33], hq=14, hkv=2, d=64, bs=128),
    "two positions": dict(ctx=[1025, 1152], spans=[2, 2], hq=4, hkv=2, d=64, bs=8),
    "mixed": dict(ctx=[300, 1, 45, 700, 260, 64, 1200], spans=[1, 1, 45, 1, 130, 2, 1], hq=16, hkv=8, d=128),
}


@pytest.mark.parametrize("name", CASES)
def test_every_key_counts_once(name):
    batch = U.Batch(seed=len(name), **CASES[name])
    each_key_of_the_bias(batch, seed=len(name))
    each_key_of_the_difference(batch)


@pytest.mark.parametrize("ctas", (1, 3, 7, 40))
def test_every_key_counts_once_in_grids(ctas):
    batch = U.Batch([1500, 3, 40, 1, 700, 90], [1] * 6, 8, 2, 64, seed=ctas)
    each_key_of_the_bias(batch, options={"decode_ctas": ctas})
    each_key_of_the_difference(batch, options={"decode_ctas": ctas})
