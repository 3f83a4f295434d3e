"""The 8-bit cache on the GPU against the fp64 oracle: append, read back, attention, and the three as
a serving step uses them.  Tolerances: tests/q8_util.py."""

import numpy as np
import pytest
import torch

import oracle
from oracle import q8 as OQ
from paged_kv_gqa_14_gb300 import _lib, ops
from tests.gpu_util import dev, dev_to_bits, idx_to_dev
from tests.q8_util import KINDS, Q8, assert_append, assert_attention, attention_tol, score_bound, value_sizes

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word():
    ops.get_device_error()
    yield
    assert ops.get_device_error() == 0, "a device error was left behind"


def raw(t):
    return t.view(torch.int8).cpu().numpy().view(np.uint8)


# -------------------------------------------------------------------------------------- append
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bs", (8, 16, 32, 64, 128))
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (16, 8, 128), (6, 3, 128), (5, 1, 64)])
def test_append_matches_oracle(kind, bs, hq, hkv, d):
    # one token, an empty span, chunks that begin and end inside blocks, a first token, a whole prompt
    c = Q8([40, 17, 300, 1, 129, 33], [1, 0, 200, 1, 129, 16], hq, hkv, d, bs, kind, seed=bs + d, extra_tokens=3,
           fresh=True).to_dev()
    c.append()
    assert_append(c, c.oracle_append())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bs", (8, 16, 128))
def test_decode_append_of_many_sequences(kind, bs):
    rng = np.random.default_rng(7)
    ctx = rng.integers(1, 300, size=1500)
    c = Q8(ctx, np.ones(1500, np.int64), 2, 1, 64, bs, kind, seed=8, fresh=True).to_dev()
    c.append()
    assert_append(c, c.oracle_append())


@pytest.mark.parametrize("kind", KINDS)
def test_steps_that_make_a_block_rescale_again_and_again(kind):
    """Decode steps of two sequences whose values grow (then shrink): each step against the oracle run on
    the state the GPU left, so that every rescaling is checked."""
    rng = np.random.default_rng(11)
    c = Q8([5, 16], [1, 1], 4, 2, 128, 16, kind, seed=12, fresh=True, num_blocks=9)
    c.bt = np.array([[4, 2, 7, -1], [0, 8, 1, -1]], np.int32)
    c.kc, c.ks = np.zeros_like(c.kc), np.ones_like(c.ks)
    c.vc, c.vs = c.kc.copy(), c.ks.copy()
    c.to_dev()
    for step in range(24):
        c.ctx = np.array([5 + step, 16 + step], np.int32)
        size = 2.0 ** (min(step, 30 - step) * 0.75)
        c.k, c.v = (oracle.f64_to_bf16_bits(rng.standard_normal((2, 2, 128)) * size) for _ in "kv")
        c.kc, c.vc = raw(c.g_kc), raw(c.g_vc)
        c.ks, c.vs = c.g_ks.cpu().numpy(), c.g_vs.cpu().numpy()
        cache = c.cache
        c.to_dev()
        c.g_kc, c.g_vc, c.g_ks, c.g_vs = cache
        ref = c.oracle_append()
        c.append()
        assert_append(c, ref)


@pytest.mark.parametrize("kind", KINDS)
def test_append_twice_changes_nothing_more(kind):
    c = Q8([50, 21], [20, 1], 4, 2, 128, 16, kind, seed=3, fresh=True).to_dev()
    q0 = c.g_q.clone()
    c.append()
    first = [t.clone() for t in c.cache]
    c.g_q.copy_(q0)
    c.append()
    for a, b in zip(first, c.cache):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("kind", KINDS)
def test_append_extremes(kind):
    """All zeros, the least scale, values at the formats' borders, bf16's largest value."""
    c = Q8([16, 16, 16, 16, 1], [16, 16, 16, 16, 1], 2, 1, 64, 16, kind, seed=4, fresh=True)
    v = np.zeros((c.T, 1, 64))
    v[16:32] = 2.0**-108
    v[32:48, 0] = np.linspace(-1, 1, 64) * OQ.LARGEST[kind]
    v[40, 0, :2] = OQ.LARGEST[kind] * 2, -0.0
    v[48:64, 0] = np.linspace(-1, 1, 64) * 3.3895313892515355e38
    v[64, 0, 5] = 0.5
    c.v = oracle.f64_to_bf16_bits(v)
    c.k = np.zeros_like(c.k)
    c.to_dev().append()
    q_rot, kc, vc, ks, vs, _ = c.oracle_append()
    top = c.bt[3, 0]
    assert np.array_equal(np.delete(raw(c.g_vc), top, 0), np.delete(vc, top, 0))
    assert np.array_equal(np.delete(c.g_vs.cpu().numpy(), top, 0), np.delete(vs.astype(np.float32), top, 0), equal_nan=True)
    assert np.array_equal(c.g_ks.cpu().numpy(), ks.astype(np.float32), equal_nan=True)
    # next to bf16's largest value the scale stays where the largest held value is finite in bf16
    s = float(c.g_vs.cpu()[top, 0])
    assert s == (2.0**121 if kind == "int8" else 2.0**119)
    held = OQ.decode(raw(c.g_vc)[top], kind)[:, 0]
    assert np.array_equal(held, OQ.decode(OQ.encode(oracle.bf16_bits_to_f64(c.v[48:64, 0]) / s, kind), kind))


@pytest.mark.parametrize("kind", KINDS)
def test_append_values_that_are_not_finite(kind):
    c = Q8([16, 20], [16, 1], 2, 1, 64, 16, kind, seed=5, fresh=True)
    c.v[3, 0, :3] = 0x7F80, 0xFF80, 0x7FC0  # inf, -inf, NaN
    c.k[4, 0, 9] = 0x7F80
    c.to_dev().append()
    assert ops.get_device_error() == 0x20
    blk = c.bt[0, 0]
    finite_v, finite_k = c.v.copy(), c.k.copy()
    finite_v[3, 0, :3] = 0
    finite_k[4, 0, [9, 41]] = 0
    c.k, c.v = finite_k, finite_v
    ref = c.oracle_append()
    got = raw(c.g_vc)
    want = ref[2].copy()
    want[blk, 3, 0, :3] = [127, 129, 0] if kind == "int8" else [0x7E, 0xFE, 0x7F]
    if kind == "e4m3":  # (a NaN's sign is the conversion's)
        assert got[blk, 3, 0, 2] & 0x7F == 0x7F
        got[blk, 3, 0, 2] = 0x7F
    assert np.array_equal(got, want)
    pair = raw(c.g_kc)[blk, 4, 0, [9, 41]]
    assert (pair == 0).all() if kind == "int8" else (pair & 0x7F == 0x7F).all()
    assert np.array_equal(c.g_ks.cpu().numpy(), ref[3].astype(np.float32), equal_nan=True)


def test_append_reads_a_packed_qkv_buffer():
    c = Q8([70, 12], [60, 1], 8, 2, 64, 16, "int8", seed=6, fresh=True).to_dev()
    packed = torch.cat([c.g_q, c.g_k, c.g_v], 1)
    c.g_q, c.g_k, c.g_v = packed[:, :8], packed[:, 8:10], packed[:, 10:]
    c.append()
    assert_append(c, c.oracle_append())


@pytest.mark.parametrize("spans", ([20, 9, 1], [1, 1, 1]))
def test_append_errors_are_flagged_and_skipped(spans):
    def run(change, bits):
        c = Q8([40, 30, 25], spans, 4, 2, 64, 16, "int8", seed=9, fresh=True)
        change(c)
        c.to_dev()
        before = [t.clone() for t in c.cache]
        c.append()
        assert ops.get_device_error() == bits
        return c, before

    def same_blocks(c, before, blocks):
        for a, b in zip(before, c.cache):
            assert torch.equal(a[blocks].view(torch.uint8), b[blocks].view(torch.uint8))

    def bad_block(c):
        c.bt[1, 1] = c.kc.shape[0]

    def short_context(c):
        c.ctx[0] = spans[0] - 1

    c, before = run(bad_block, 0x2)
    c, before = run(short_context, 0x4)
    same_blocks(c, before, c.bt[0, :3].tolist())

    c = Q8([40, 30, 25], spans, 4, 2, 64, 16, "int8", seed=9, fresh=True).to_dev()
    before = [t.clone() for t in c.cache]
    c.append(max_blocks_per_seq=2)  # sequence 0's tokens in block 2 (and only they) have no place
    assert ops.get_device_error() == 0x8
    same_blocks(c, before, [int(c.bt[0, 2])])


# ---------------------------------------------------------------------------------------- read
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hkv,d,bs", [(1, 64, 8), (2, 64, 16), (8, 128, 16), (3, 128, 64), (4, 64, 128)])
def test_read_is_exact(kind, hkv, d, bs):
    ctx = [1, 40, 17, 300, 64]
    c = Q8(ctx, [1] * 5, hkv, hkv, d, bs, kind, seed=d + bs).to_dev()
    k = OQ.dequantise(c.kc, c.ks, kind)
    v = OQ.dequantise(c.vc, c.vs, kind)
    for lens in (ctx, [1, 0, 5, 123, 0]):
        rsl = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        rows = int(rsl[-1]) + 2
        outs = [torch.full((rows, hkv, d), 7.0, dtype=torch.bfloat16, device=dev()) for _ in "kv"]
        ops.kv_read_q8(*c.cache, c.g_bt, c.g_ctx, idx_to_dev(rsl), *outs)
        for pool, out in zip((k, v), outs):
            want = np.full((rows, hkv, d), 0x40E0, np.uint16)  # 7.0: left as it was
            for b, n in enumerate(lens):
                p = np.arange(ctx[b] - n, ctx[b])
                want[rsl[b]:rsl[b + 1]] = pool[c.bt[b, p // bs], p % bs]
            assert np.array_equal(dev_to_bits(out), want)


def test_read_into_strided_outputs_and_errors():
    c = Q8([40, 30], [1, 1], 2, 2, 64, 16, "e4m3", seed=1).to_dev()
    rsl = idx_to_dev(np.array([0, 40, 70], np.int32))
    want = [torch.empty(70, 2, 64, dtype=torch.bfloat16, device=dev()) for _ in "kv"]
    ops.kv_read_q8(*c.cache, c.g_bt, c.g_ctx, rsl, *want)
    both = torch.zeros(2, 2, 70, 128, dtype=torch.bfloat16, device=dev())  # head-major, rows of 128
    views = [x.transpose(0, 1)[..., 64:] for x in both]
    ops.kv_read_q8(*c.cache, c.g_bt, c.g_ctx, rsl, *views)
    assert all(torch.equal(a, b) for a, b in zip(want, views)) and not both[..., :64].any()
    table = c.g_bt.clone()
    table[1, 0] = -1
    out = [torch.zeros_like(x) for x in want]
    ops.kv_read_q8(*c.cache, table, c.g_ctx, rsl, *out)
    assert ops.get_device_error() == 0x2
    assert not out[0][40:56].any() and torch.equal(out[0][56:], want[0][56:]) and torch.equal(out[1][:40], want[1][:40])
    ops.kv_read_q8(*c.cache, c.g_bt, c.g_ctx, rsl, *out, max_blocks_per_seq=2)
    assert ops.get_device_error() == 0x8
    ops.kv_read_q8(*c.cache, c.g_bt, c.g_ctx, idx_to_dev(np.array([0, 41, 70], np.int32)), *out)
    assert ops.get_device_error() == 0x4


# ----------------------------------------------------------------------------------- attention
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bs", (8, 16, 32, 64, 128))
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("hkv", (1, 2, 4, 8))
def test_decode_matches_oracle(kind, bs, d, hkv):
    group = 1 + (bs + hkv + d // 64) % 8
    rng = np.random.default_rng(bs * hkv + d)
    ctx = np.concatenate([[1, 2, 7, 8, 9, 15, 16, 17, 127, 128, 129], rng.integers(1, 500, size=5)])
    c = Q8(ctx, np.ones(len(ctx), np.int64), hkv * group, hkv, d, bs, kind, seed=hkv + d + bs).to_dev()
    ref, tol = c.oracle_attention()
    assert_attention(c.attend(), ref, tol)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("group", range(1, 9))
@pytest.mark.parametrize("d,bs", [(64, 16), (128, 8), (128, 64)])
def test_prefill_matches_oracle(kind, group, d, bs):
    ctx, spans = [300, 129, 2, 140, 513], [140, 129, 2, 3, 33]
    c = Q8(ctx, spans, 2 * group, 2, d, bs, kind, seed=group + d).to_dev()
    ref, tol = c.oracle_attention()
    assert_attention(c.attend(), ref, tol)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("overlap", (None, False))
@pytest.mark.parametrize("seed", range(4))
def test_mixed_batches(kind, overlap, seed):
    rng = np.random.default_rng(100 + seed)
    hkv, d, bs = int(rng.choice([1, 2, 4, 8])), int(rng.choice([64, 128])), int(rng.choice([8, 16, 32, 64, 128]))
    n = 24
    ctx = rng.integers(1, 600, size=n)
    spans = np.where(rng.random(n) < 0.5, 1, rng.integers(0, 1 + np.minimum(ctx, 150)))
    c = Q8(ctx, spans, hkv * int(rng.integers(1, 9)), hkv, d, bs, kind, seed=seed, extra_tokens=2).to_dev()
    out = torch.full_like(c.g_q, 3.0)
    c.attend(out=out, options={"overlap": overlap})
    ref, tol = c.oracle_attention()
    covered = np.arange(c.T) < c.qsl[-1]
    assert_attention(out, ref, tol, covered)
    assert (out[~torch.from_numpy(covered).to(dev())] == 3.0).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,bs", [(64, 8), (128, 16), (128, 128)])
@pytest.mark.parametrize("ctx,spans,hq,hkv", [
    ([1500], [37], 2, 1),  # one item: twelve key tiles, so that the last pieces are empty
    ([130], [3], 7, 1),
    ([1153], [2], 8, 8),
    ([200], [200], 4, 4),  # the second piece's keys are past the first Q tile's rows
    ([700, 650, 129, 1, 900, 333, 40], [5, 64, 129, 1, 2, 70, 40], 12, 4),
    ([90 + 17 * i for i in range(25)], [2] * 25, 5, 1),
    ([90 + 9 * i for i in range(30)], [3] * 30, 2, 2),
    ([300, 1, 140] * 34, [2, 1, 3] * 34, 2, 2),  # more items than would be shared
])
def test_few_prefill_items_are_shared_among_ctas(kind, d, bs, ctx, spans, hq, hkv):
    c = Q8(ctx, spans, hq, hkv, d, bs, kind, seed=len(ctx) + d, extra_tokens=1).to_dev()
    ref, tol = c.oracle_attention()
    covered = np.arange(c.T) < c.qsl[-1]
    for options in (None, {"overlap": False}):
        out = torch.full_like(c.g_q, 3.0)
        c.attend(out=out, options=options)
        assert_attention(out, ref, tol, covered)
        assert (out[~torch.from_numpy(covered).to(dev())] == 3.0).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bs", (8, 16))
def test_blocks_whose_scales_lie_far_apart(kind, bs):
    """V scales of 2^-40 to 2^40 from block to block (decode) and 2^-9 to 2^9 (prefill tiles too): the
    allowed error is relative to the weighted |V|, which small blocks dominate where large ones are masked."""
    c = Q8([300, 257, 90], [1, 1, 1], 8, 4, 128, bs, kind, seed=2)
    rng = np.random.default_rng(3)
    c.vs = np.where(np.isnan(c.vs), c.vs, np.ldexp(1.0, rng.integers(-40, 41, size=c.vs.shape))).astype(np.float32)
    c.to_dev()
    ref, tol = c.oracle_attention()
    assert_attention(c.attend(), ref, tol)
    c = Q8([300, 257, 90], [200, 257, 1], 8, 4, 128, bs, kind, seed=2)
    for s in (c.ks, c.vs):
        s[:] = np.where(np.isnan(s), s, np.ldexp(1.0, rng.integers(-9, 10, size=s.shape)))
    c.q = oracle.f64_to_bf16_bits(oracle.bf16_bits_to_f64(c.q) * 2.0**-9)
    c.to_dev()
    ref, tol = c.oracle_attention()
    assert_attention(c.attend(), ref, tol)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("spans", ([1, 1], [1, 1, 5]))
def test_one_key_gives_its_value(kind, spans):
    """A row that sees one key returns the value the cache stands for, bit for bit."""
    c = Q8([1, 1, 5][: len(spans)], spans, 4, 2, 64, 16, kind, seed=1).to_dev()
    v = OQ.dequantise(c.vc, c.vs, kind)
    got = dev_to_bits(c.attend())
    for b in range(len(spans)):
        want = np.repeat(v[c.bt[b, 0], 0], 2, axis=0)
        zero = oracle.bf16_bits_to_f64(want) == 0  # (a zero's sign is lost)
        assert ((got[c.qsl[b]] == want) | (zero & (got[c.qsl[b]] & 0x7FFF == 0))).all()


@pytest.mark.parametrize("kind", KINDS)
def test_zero_and_huge_queries(kind):
    """Zero queries (the mean of the visible values, all-zero keys among them), queries of 2^60 and 2^-60."""
    c = Q8([100, 100, 100, 130], [1, 1, 1, 64], 4, 2, 64, 16, kind, seed=1)
    x = oracle.bf16_bits_to_f64(c.q)
    x[0] = 0.0
    x[1] *= 2.0**60
    x[2] *= 2.0**-60
    x[3:35] = 0.0
    x[35:] *= 2.0**-60
    c.q = oracle.f64_to_bf16_bits(x)
    blk = c.bt[1, : 7]
    c.ks[blk] = 2.0**-62  # keeps the scores of the huge query in range
    z = c.bt[3, : 9]
    c.kc[z], c.ks[z] = 0, 2.0**-100
    c.to_dev()
    # scores are small, but |q| |k| over the whole batch is not: bound them by sequence
    ref, _ = c.oracle_attention()
    k, v = OQ.dequantise(c.kc, c.ks, kind), OQ.dequantise(c.vc, c.vs, kind)
    size, total = value_sizes(c.q, k, v, c.bt, c.ctx, c.qsl, c.scale)
    tol = np.empty_like(ref)
    for b in range(4):
        r = slice(int(c.qsl[b]), int(c.qsl[b + 1]))
        tol[r] = attention_tol(ref[r], size[r], total[r], score_bound(c.q[r], k, c.bt[b:b + 1], c.ctx[b:b + 1], c.scale))
    assert_attention(c.attend(), ref, tol)


def test_nan_and_infinite_scores_stay_in_their_rows():
    """A NaN in one query's row and in one sequence's keys makes only those rows NaN."""
    c = Q8([40, 40, 60, 60], [1, 1, 20, 20], 4, 2, 64, 16, "e4m3", seed=1)
    c.q[0, 1, 3] = 0x7FC0
    c.kc[c.bt[1, 1], 2, 1, 7] = 0x7F
    c.q[2 + 5, 2, 0] = 0x7FC0
    c.to_dev()
    got = c.attend().float().cpu().numpy()
    bad = np.zeros((c.T, 4), bool)
    bad[0, 1] = True
    bad[1, 2:] = True
    bad[7, 2] = True
    assert np.array_equal(np.isnan(got).all(-1), bad) and np.array_equal(np.isnan(got).any(-1), bad)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hkv,d,bs", [(8, 128, 16), (1, 64, 8), (2, 128, 128)])
def test_a_long_context_split_over_every_cta(kind, hkv, d, bs):
    c = Q8([5000, 3], [1, 1], 2 * hkv, hkv, d, bs, kind, seed=1, spread=1).to_dev()
    ref, tol = c.oracle_attention()
    assert_attention(c.attend(), ref, tol)
    for ctas in (1, 2, 7, 300):
        assert_attention(c.attend(options={"decode_ctas": ctas}), ref, tol)


@pytest.mark.parametrize("kind", KINDS)
def test_rows_of_longer_spans_without_more_tokens_than_sequences(kind):
    c = Q8([50, 20, 33, 9, 70], [3, 0, 1, 0, 1], 4, 2, 128, 16, kind, seed=1).to_dev()
    ref, tol = c.oracle_attention()
    assert_attention(c.attend(), ref, tol)


@pytest.mark.parametrize("options", (None, {"plan_early": True}, {"stream_early": True}))
def test_more_sequences_than_threads_plan(options):
    """Batches past one scan of a CTA's threads, with empty and (seldom) longer spans among them."""
    rng = np.random.default_rng(1)
    ctx = rng.integers(1, 40, size=1300)
    spans = np.ones(1300, np.int64)
    spans[rng.integers(0, 1300, size=60)] = 0
    spans[700] = min(7, ctx[700])
    c = Q8(ctx, spans, 2, 1, 64, 8, "int8", seed=1).to_dev()
    ref, tol = c.oracle_attention()
    assert_attention(c.attend(options=options), ref, tol)


def test_nothing_to_attend_to():
    """Spans that are all in error or empty: every row is left, and the next call runs as ever."""
    c = Q8([40, 30, 20], [1, 1, 1], 4, 2, 64, 16, "int8", seed=1).to_dev()
    want = c.attend()
    out = torch.full_like(c.g_q, 2.0)
    ctx, c.g_ctx = c.g_ctx, torch.zeros_like(c.g_ctx)
    for options in (None, {"plan_early": True}, {"stream_early": True}):
        c.attend(out=out, options=options)
        assert ops.get_device_error() == 0x4 and (out == 2.0).all()
    c.g_ctx, qsl, c.g_qsl = ctx, c.g_qsl, torch.zeros_like(c.g_qsl)
    c.attend(out=out)
    assert (out == 2.0).all()
    c.g_qsl = qsl
    assert torch.equal(c.attend(out=out), want)


def test_strided_q_and_out_and_a_query_shared_by_rows():
    c = Q8([90, 40], [30, 1], 4, 2, 64, 16, "int8", seed=1).to_dev()
    want = c.attend()
    wide = torch.zeros(c.T, 9, 64, dtype=torch.bfloat16, device=dev())
    wide[:, 2:6] = c.g_q
    out = torch.full((4, c.T, 128), 5.0, dtype=torch.bfloat16, device=dev())  # head-major
    view = out.transpose(0, 1)[..., :64]
    q0, c.g_q = c.g_q, wide[:, 2:6]
    c.attend(out=view)
    assert torch.equal(view, want) and (out[..., 64:] == 5.0).all()
    c.g_q = q0[:1].expand(c.T, 4, 64)  # stride 0 over tokens
    got = c.attend()
    c.g_q = c.g_q.contiguous()
    assert torch.equal(got, c.attend())


def test_attention_errors_are_flagged():
    def run(bits, change):
        c = Q8([40, 300, 60], [1, 200, 1], 4, 2, 64, 16, "int8", seed=1)
        change(c)
        c.to_dev().attend()
        assert ops.get_device_error() == bits

    def block(c):
        c.bt[0, 1] = 10**6
        c.bt[1, 2] = -5

    def span(c):
        c.ctx[1] = 100

    run(0x2, block)
    run(0x4, span)
    c = Q8([40, 300, 60], [1, 200, 1], 4, 2, 64, 16, "int8", seed=1).to_dev()
    c.attend(max_blocks_per_seq=4)
    assert ops.get_device_error() == 0x8


def test_the_binding_refuses_before_any_launch():
    c = Q8([40], [1], 4, 2, 64, 16, "int8", seed=1).to_dev()
    ws = ops.alloc_workspace(1, 1, 4, 2, 64, c.bt.shape[1])
    with pytest.raises(_lib.PkvError, match="WORKSPACE"):
        c.attend(workspace=ws[:256])
    with pytest.raises(_lib.PkvError, match="UNSUPPORTED"):
        c.attend(options={"decode_kernel": "simt"})
    with pytest.raises(ValueError, match="block_tables"):
        c.attend(max_blocks_per_seq=99)
    with pytest.raises(ValueError, match="scale"):
        ops.paged_attention_q8(c.g_q, c.g_kc, c.g_vc, c.g_ks[:-1], c.g_vs, c.g_bt, c.g_ctx, c.g_qsl, 0.1)
    with pytest.raises(TypeError):
        ops.paged_attention_q8(c.g_q, c.g_kc, c.g_vc.view(torch.float8_e4m3fn), c.g_ks, c.g_vs, c.g_bt, c.g_ctx, c.g_qsl, 0.1)
    with pytest.raises(ValueError, match="CUDA|cpu"):
        ops.paged_attention_q8(c.g_q, c.g_kc, c.g_vc, c.g_ks, c.g_vs, c.g_bt, c.g_ctx.cpu(), c.g_qsl, 0.1)


def test_bounded_waits_run_out_and_report():
    c = Q8([200, 100], [1, 1], 4, 2, 64, 16, "int8", seed=1).to_dev()
    want = c.attend()
    ops.set_fault_injection("decode_no_copies")
    try:
        c.attend()
        assert ops.get_device_error() == 0x10
    finally:
        ops.set_fault_injection(None)
    assert torch.equal(c.attend(), want)


def test_a_pool_past_2_31_bytes():
    """Blocks whose bytes lie past 2^31 (and 2^32) in each pool, written, read and attended."""
    nb, bs, hkv, d = 300_000, 16, 8, 128
    kc, vc, ks, vs = ops.alloc_q8_cache(nb, bs, hkv, d)
    assert kc.numel() > 1 << 32
    c = Q8([100, 40], [60, 1], 16, hkv, d, bs, "int8", seed=1, fresh=True, num_blocks=12)
    place = np.array([nb - 1, 5, nb - 2, 131072 * 2 + 1, 262144, nb - 3, 0, nb // 2, 140000, 270001, nb - 9, 17])
    c.to_dev()
    at = torch.from_numpy(place).to(dev())
    for big, small in zip((kc, vc, ks, vs), c.cache):
        big[at] = small
    far = idx_to_dev(np.where(c.bt >= 0, place[np.maximum(c.bt, 0)], -1).astype(np.int32))
    q2 = c.g_q.clone()
    c.append()
    want = c.attend()
    ops.kv_append_q8(q2, c.g_k, c.g_v, far, c.g_ctx, c.g_qsl, kc, vc, ks, vs, c.theta)
    for big, small in zip((kc, vc, ks, vs), c.cache):
        assert torch.equal(big[at].view(torch.uint8), small.view(torch.uint8))
    got = ops.paged_attention_q8(q2, kc, vc, ks, vs, far, c.g_ctx, c.g_qsl, c.scale)
    assert torch.equal(got, want)
    rsl = idx_to_dev(np.array([0, 100, 140], np.int32))
    outs = [[torch.empty(140, hkv, d, dtype=torch.bfloat16, device=dev()) for _ in "kv"] for _ in "ab"]
    ops.kv_read_q8(kc, vc, ks, vs, far, c.g_ctx, rsl, *outs[0])
    ops.kv_read_q8(*c.cache, c.g_bt, c.g_ctx, rsl, *outs[1])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


# -------------------------------------------------------------------------------- the step
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("options", (None, {"plan_early": True}, {"stream_early": True},
                                     {"stream_early": True, "overlap": False}))
@pytest.mark.parametrize("bs", (8, 16, 128))
def test_step_append_attention_read(kind, options, bs):
    """A step as an engine runs it, back to back on one stream: the attention sees what the append
    wrote, whatever it may start early; the read gives what the attention saw."""
    rng = np.random.default_rng(3)
    ctx = rng.integers(1, 900, size=40)
    spans = np.ones(40, np.int64)
    spans[:3] = np.minimum(ctx[:3], 90)
    c = Q8(ctx, spans, 8, 2, 64, bs, kind, seed=5, fresh=True).to_dev()
    start = [t.clone() for t in (c.g_q, *c.cache)]
    ws = ops.alloc_workspace(c.T, 40, 8, 2, 64, c.bt.shape[1])
    opt = ops.attention_options(options)
    for _ in range(3):
        for t, s in zip((c.g_q, *c.cache), start):
            t.copy_(s)
        c.append()
        out = c.attend(workspace=ws, options=opt)
    kc, vc, ks, vs = raw(c.g_kc), raw(c.g_vc), c.g_ks.cpu().numpy(), c.g_vs.cpu().numpy()
    ref, tol = c.oracle_attention(dev_to_bits(c.g_q), kc, vc, ks, vs)
    assert_attention(out, ref, tol)
    rsl = np.concatenate([[0], np.cumsum(ctx)]).astype(np.int32)
    k, v = (torch.empty(int(rsl[-1]), 2, 64, dtype=torch.bfloat16, device=dev()) for _ in "kv")
    ops.kv_read_q8(*c.cache, c.g_bt, c.g_ctx, idx_to_dev(rsl), k, v)
    want = np.concatenate([OQ.dequantise(kc, ks, kind)[c.bt[b, np.arange(n) // bs], np.arange(n) % bs]
                           for b, n in enumerate(ctx)])
    assert np.array_equal(dev_to_bits(k), want)


def test_step_in_a_graph_and_on_another_stream():
    c = Q8([200, 64, 33, 500], [1, 1, 1, 100], 8, 4, 128, 16, "int8", seed=5, fresh=True).to_dev()
    start = [t.clone() for t in (c.g_q, *c.cache)]
    state = (c.g_q, *c.cache)
    ws = ops.alloc_workspace(c.T, 4, 8, 4, 128, c.bt.shape[1])
    out = torch.empty_like(c.g_q)
    rsl = idx_to_dev(np.concatenate([[0], np.cumsum(c.ctx)]).astype(np.int32))
    k, v = (torch.empty(int(c.ctx.sum()), 4, 128, dtype=torch.bfloat16, device=dev()) for _ in "kv")

    def step(stream=None):
        c.append(stream=stream)
        c.attend(out=out, workspace=ws, stream=stream)
        ops.kv_read_q8(*c.cache, c.g_bt, c.g_ctx, rsl, k, v, stream=stream)

    def reset():
        for t, s in zip(state, start):
            t.copy_(s)
        out.zero_(), k.zero_(), v.zero_()

    step()
    want = [t.clone() for t in (out, k, v, *state)]
    side = torch.cuda.Stream()
    reset()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, (out, k, v, *state)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    g = torch.cuda.CUDAGraph()
    reset()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        reset()
        g.replay()
        for a, b in zip(want, (out, k, v, *state)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_two_calls_at_once():
    """Mixed batches on two streams, each with its workspace: the library's second stream serves both."""
    cs = [Q8([700, 90, 33, 500], spans, 8, 4, 128, 16, "int8", seed=s).to_dev()
          for s, spans in ((5, [1, 60, 1, 100]), (6, [300, 1, 33, 1]))]
    wss = [ops.alloc_workspace(c.T, 4, 8, 4, 128, c.bt.shape[1]) for c in cs]
    want = [c.attend(workspace=w) for c, w in zip(cs, wss)]
    outs = [[torch.zeros_like(w) for _ in range(6)] for w in want]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for i in range(6):
        for c, w, o, s in zip(cs, wss, outs, streams):
            c.attend(out=o[i], workspace=w, stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, x) for x in o)


@pytest.mark.parametrize("ctx", ([100, 7, 64, 31], [3000, 2, 900]))
def test_graphs_that_share_a_workspace_and_calls_between_them(ctx):
    """Pieces merged in the decode kernel and by the one after it: the words they count and leave in the workspace
    disturb neither a replay of another graph nor a bf16 call."""
    n = len(ctx)
    cs = [Q8(ctx, [1] * n, 16, 8, 64, 16, "int8", seed=s).to_dev() for s in (1, 2)]
    ws = ops.alloc_workspace(n, n, 16, 8, 64, cs[0].bt.shape[1])
    outs = [torch.empty_like(c.g_q) for c in cs]
    kb, vb = (torch.randn(*cs[0].g_kc.shape, device=dev()).to(torch.bfloat16) for _ in "kv")

    def plain():
        return ops.paged_attention(cs[0].g_q, kb, vb, cs[0].g_bt, cs[0].g_ctx, cs[0].g_qsl, cs[0].scale, workspace=ws)

    want = [c.attend(workspace=ws).clone() for c in cs]
    want_plain = plain()
    graphs = []
    for c, o in zip(cs, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c.attend(out=o, workspace=ws)
    for i in (0, 1, 1, 0, 1, 0):
        outs[i].zero_()
        graphs[i].replay()
        assert torch.equal(outs[i], want[i])
        assert torch.equal(plain(), want_plain)


@pytest.mark.parametrize("group,ctas", [(8, 0), (8, 2), (8, 40), (1, 0), (3, 152)])
def test_pieces_of_many_columns_and_of_few(group, ctas):
    c = Q8([4100, 60, 1500], [1, 1, 1], 8 * group, 8, 128, 16, "e4m3", seed=group, spread=1).to_dev()
    ref, tol = c.oracle_attention()
    assert_attention(c.attend(options={"decode_ctas": ctas} if ctas else None), ref, tol)


@pytest.mark.parametrize("hq,hkv,bs", [(200, 200, 32), (1024, 1024, 16)])
def test_append_of_many_heads(hq, hkv, bs):
    c = Q8([40, 9, 1], [21, 9, 1], hq, hkv, 64, bs, "int8", seed=hkv, fresh=True).to_dev()
    ref = c.oracle_append()
    c.append()
    assert_append(c, ref)


@pytest.mark.parametrize("hkv,d,n", [(1, 64, 70001), (2, 128, 40003), (3, 64, 300007)])
def test_read_of_many_rows(hkv, d, n):
    """Calls large enough that a warp takes four and eight pieces to a lane: three ranges, one of them empty."""
    bs, lens = 16, [n, 0, n // 3]
    nb = [-(-x // bs) for x in lens]
    g = torch.Generator(device=dev()).manual_seed(n)
    perm = torch.randperm(sum(nb), generator=g, device=dev()).to(torch.int32)
    table = torch.full((3, max(nb)), -1, dtype=torch.int32, device=dev())
    table[0, : nb[0]], table[2, : nb[2]] = perm[: nb[0]], perm[nb[0]:]
    kc, vc = (torch.randint(-127, 128, (sum(nb), bs, hkv, d), dtype=torch.int8, generator=g, device=dev()) for _ in "kv")
    ks, vs = ((torch.randint(118, 137, (sum(nb), hkv), dtype=torch.int32, generator=g, device=dev()) << 23)
              .view(torch.float32) for _ in "kv")  # 2^-9 .. 2^9
    rsl = idx_to_dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    out = [torch.zeros(sum(lens) + 5, hkv, d, dtype=torch.bfloat16, device=dev()) for _ in "kv"]
    ops.kv_read_q8(kc, vc, ks, vs, table, idx_to_dev(np.array(lens, np.int32)), rsl, *out)
    for o, c, s in ((out[0], kc, ks), (out[1], vc, vs)):
        at = 0
        for b in (0, 2):
            blocks = table[b, : nb[b]].long()
            want = (c[blocks].float() * s[blocks][:, None, :, None]).view(-1, hkv, d)[: lens[b]].to(torch.bfloat16)
            assert torch.equal(o[at : at + lens[b]], want)
            at += lens[b]
        assert not o[at:].any()
    assert ops.get_device_error() == 0
