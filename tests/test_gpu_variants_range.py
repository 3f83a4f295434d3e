"""The attention variants at the ends of what scores, values and lengths may be."""

import numpy as np
import pytest
import torch

import oracle
from oracle import variants as OV
from paged_kv_gqa_14_gb300 import ops
from tests import variants_util as U

pytestmark = pytest.mark.gpu

T5 = (32, 128)
HALF_BF16 = OV.HALF_BF16


# ------------------------------------------------------------------------------- large scores
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("power", (10, 17, 20, 23, 24, 25, 27, 30, 40, 80))
@pytest.mark.parametrize("sign", (1, -1))
def test_scores_past_what_fp32_holds_to_a_unit(d, power, sign):
    """Scores of 2^13 to 2^90 (all of them positive, or negative): the largest by far takes all of the softmax.  It is
    key 0's until, from key 150 on, a larger one.  Decode rows and prefill rows, the latter's items shared or not."""
    for spans, ctx in (([1, 1, 200], [300, 120, 280]), ([12, 1], [2000, 30]), ([250] * 12 + [1], [290] * 13)):
        c = U.Batch(ctx, spans, 16, 8, d, seed=power)
        q = np.sign(oracle.bf16_bits_to_f64(c.q[0, ::2])) * (1 + np.arange(d) / 128)  # [hkv, d], exact in bf16
        q[q == 0] = 1
        way = np.sign(q)
        c.q = oracle.f64_to_bf16_bits(np.repeat(np.repeat(q, 2, 0)[None], c.T, 0) * 2.0**power)
        rng = np.random.default_rng(power)
        bt = c.bt.block_tables
        sizes = []
        for b, n in enumerate(ctx):
            size = rng.integers(1, 12, n).astype(float)
            size[0], size[150:151] = 30.0, 112.0
            if sign < 0:
                size = np.where(size == 30.0, -28.0, np.where(size == 112.0, -2.0, size - 100.0))
            sizes.append(size)
            for p in range(n):
                c.kc[bt[b, p // 16], p % 16] = oracle.f64_to_bf16_bits(way * size[p])
        args = c.dev()
        bias, buckets = torch.zeros(32, 16, device="cuda"), ops.relative_buckets(*T5)
        lam = np.linspace(0.25, 0.75, 8).astype(np.float32)
        v = oracle.bf16_bits_to_f64(c.vc)
        for options in (None, {"overlap": False}):
            plain = ops.paged_attention_bias(*args, bias, buckets, options=options).double().cpu().numpy()
            # q heads 2h and 2h + 1 of the pair's two maps: q heads 4g .. 4g + 3 are k heads 2g, 2g, 2g + 1, 2g + 1
            # of the plain layout; here head h uses k heads 2 (h // 2) and 2 (h // 2) + 1
            dq = args[0].view(c.T, 4, 2, 2, d).transpose(2, 3).reshape(c.T, 16, d).contiguous()
            diff = ops.paged_attention_diff(dq, *args[1:], torch.from_numpy(lam).cuda(), options=options)
            diff = diff.double().cpu().numpy()
            assert ops.get_device_error() == 0
            at = 0
            for b, n in enumerate(ctx):
                for r in range(spans[b]):
                    key = 150 if n - spans[b] + r >= 150 else 0
                    row = v[bt[b, key // 16], key % 16]  # [hkv, d]
                    # one key of weight 1: its value, which bf16 holds
                    assert np.array_equal(plain[at], np.repeat(row, 2, axis=0)), (b, r)
                    # (1 - lam) v, rounded once after fp32 sums
                    want = (1 - lam.astype(np.float64))[:, None] * np.repeat(row.reshape(4, 2 * d), 2, axis=0)
                    assert np.all(np.abs(diff[at] - want) <= (HALF_BF16 + 2.0**-20) * np.abs(want)), (b, r)
                    at += 1


# -------------------------------------------------------------------------------- large values
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("power", (60, 100, 112))
def test_large_values_behind_low_scores(d, power):
    """V of 2^112 and, after 150 keys of low scores, keys that score just below 2^20 times their weight: sums of 2^11
    weights stay inside fp32 when no weight is above 1, and would not if one could be 2^20."""
    for spans, ctx in (([1, 1, 200], [2000, 300, 1900]), ([12, 1], [2000, 30]), ([250] * 12 + [1], [290] * 12 + [1700])):
        c = U.Batch(ctx, spans, 8, 4, d, seed=power, scale=0.125)
        q = np.zeros((c.T, 8, d))
        q[:, :, 0] = 1.0
        c.q = oracle.f64_to_bf16_bits(q)
        rng = np.random.default_rng(power)
        bt = c.bt.block_tables
        for b, n in enumerate(ctx):
            for p in range(n):
                k = np.zeros((4, d))
                k[:, 0] = 0.0 if p < 150 else 110.0  # log2 of the weight: 110 x 0.125 x log2(e) = 19.84
                c.kc[bt[b, p // 16], p % 16] = oracle.f64_to_bf16_bits(k)
                c.vc[bt[b, p // 16], p % 16] = oracle.f64_to_bf16_bits(rng.uniform(1, 2, (4, d)) * 2.0**power)
        buckets, bias = ops.relative_buckets(*T5), torch.zeros(32, 8)
        U.check_bias(c, buckets, bias, bias.double().numpy(), OV.log_starts(*T5), what=f"bias {spans[0]}")
        U.check_diff(c, np.full(4, 0.5, np.float32), what=f"diff {spans[0]}")


# ------------------------------------------------------------------------------ another stream
def _calls_on(c, zero):
    """The attentions of a batch, as functions of the pool's values (``zero`` or others) and of what a call may be
    given."""
    q, kc, vc, bt, ctx, qsl, scale = c.dev()
    lam, bias, buckets = torch.full((c.hq // 2,), 0.5, device="cuda"), torch.zeros(32, c.hq, device="cuda"), ops.relative_buckets(*T5)
    k8, v8, ks, vs = ops.alloc_q8_cache(*kc.shape)
    for x, n in ((k8, 1), (v8, 3), (ks, 1), (vs, 1)):
        x.fill_(n)
    zero8 = torch.zeros_like(v8)
    return {"plain": lambda v, **kw: ops.paged_attention(q, kc, v, bt, ctx, qsl, scale, **kw),
            "bias": lambda v, **kw: ops.paged_attention_bias(q, kc, v, bt, ctx, qsl, scale, bias, buckets, **kw),
            "diff": lambda v, **kw: ops.paged_attention_diff(q, kc, v, bt, ctx, qsl, scale, lam, **kw),
            "q8": lambda v, **kw: ops.paged_attention_q8(q, k8, zero8 if v is zero else v8, ks, vs, bt, ctx, qsl, scale, **kw)}


@pytest.mark.parametrize("name", ("plain", "bias", "diff", "q8"))
def test_an_output_made_for_another_stream_waits_for_both(name):
    """An output that is not given must not be memory that the current stream still reads, and must not be given to
    the next call on the other stream while the current one still reads it."""
    c = U.Batch([4096], [4096], 16, 8, 64, seed=3)
    vc = c.dev()[2].nan_to_num(0.0)
    zero = torch.zeros_like(vc)
    call = _calls_on(c, zero)[name]
    side = torch.cuda.Stream()
    want = call(vc)
    call(vc, stream=side)  # (its workspace is kept for the other stream)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    x = torch.ones(want.shape, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # (about 50 ms)
    y.copy_(x)
    del x
    out = call(vc, stream=side)
    torch.cuda.synchronize()
    assert bool((y == 1).all()) and torch.equal(out, want)
    torch.cuda._sleep(100_000_000)
    y.copy_(out)
    del out
    again = call(zero, stream=side)
    again2 = call(zero, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    assert torch.equal(again, call(zero)) and torch.equal(again2, again)
    assert ops.get_device_error() == 0


# ---------------------------------------------------------------------------------- alike maps
def _alike(c, corr):
    """Makes the second map's queries and keys those of the first but for a part of 1 - corr^2."""
    q, kc = oracle.bf16_bits_to_f64(c.q), oracle.bf16_bits_to_f64(c.kc)
    rest = np.sqrt(1 - corr * corr)
    q[:, 1::2] = corr * q[:, 0::2] + rest * q[:, 1::2]
    kc[:, :, 1::2] = corr * kc[:, :, 0::2] + rest * kc[:, :, 1::2]
    held = ~np.isnan(kc)
    c.q = oracle.f64_to_bf16_bits(q)
    c.kc[held] = oracle.f64_to_bf16_bits(np.where(held, kc, 0.0))[held]
    return c


@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("corr", (0.9, 0.99))
@pytest.mark.parametrize("lam", (0.8, 1.0))
def test_decode_of_the_difference_of_alike_maps(d, corr, lam):
    """What two maps share drops out and the norm scales the rest up again: weights rounded to bf16 alone would show.  The
    decode multiplies with two bf16 parts of a weight, whose sum is off by at most 2^-9 of a half step of 2^-8."""
    ctx = [2, 3, 5, 8, 12, 16, 17, 24, 31, 40, 200, 700]
    c = _alike(U.Batch(ctx, [1] * len(ctx), 8, 4, d, seed=d), corr)
    lam = np.full(4, lam, np.float32)
    for weight in (None, U.weight_of(c, 1)):
        ref, slack = OV.paged_attention_diff(*c.host(), lam, weight, weight_error=2.0**-17)
        out = U.marked(c.T, 4, 2 * d)
        for options in (None, {"decode_ctas": 3}):  # (entries whole, and in pieces)
            ops.paged_attention_diff(*c.dev(), torch.from_numpy(lam).cuda(), out=out, options=options,
                                     norm_weight=None if weight is None else torch.from_numpy(weight).cuda())
            torch.cuda.synchronize()
            U.within(out, ref, slack, f"norm {weight is not None}")
    assert ops.get_device_error() == 0


@pytest.mark.parametrize("d", (64, 128))
def test_prefill_of_the_difference_of_alike_maps(d):
    """One bf16 part: within what that may lose of each map, whatever the difference leaves of the maps."""
    c = _alike(U.Batch([30, 400, 1500], [30, 70, 9], 8, 4, d, seed=d + 1), 0.99)
    for weight in (None, U.weight_of(c, 1)):
        U.check_diff(c, np.full(4, 1.0, np.float32), weight, what=f"norm {weight is not None}")


@pytest.mark.parametrize("name", ("bias", "diff"))
def test_captured_calls_on_another_stream_make_their_own_output(name):
    c = U.Batch([300, 77, 200], [1, 77, 60], 8, 2, 64, seed=65)
    vc = c.dev()[2]
    call, side = _calls_on(c, None)[name], torch.cuda.Stream()
    want = call(vc)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        outs = [call(vc, stream=side) for _ in range(3)]
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for out in outs:
            out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for out in outs)
    assert ops.get_device_error() == 0


# ------------------------------------------------------------------- joins inside a captured decode
def test_replays_that_join_pieces_in_the_decode():
    """Small batches whose pieces are joined by the CTA that writes the last one: a counter in the workspace, tagged by the
    captured call, ends each replay as it began, also when calls that lay the workspace out otherwise come between."""
    dec = U.Batch([900, 64, 513, 130], [1] * 4, 8, 2, 64, seed=61)  # 8 units of 128 keys, and fewer
    one = U.Batch([700], [1], 4, 2, 64, seed=62)  # one entry in several pieces
    mix = U.Batch([300, 77, 200], [1, 77, 60], 8, 2, 64, seed=63)  # planned by a kernel of its own
    buckets = ops.relative_buckets(*T5)
    ws = ops.alloc_workspace(mix.T, 4, 8, 2, 64, 64, diff=True)
    calls, outs, wants, graphs = [], [], [], []
    for batch in (dec, one, mix):
        args = batch.dev()
        lam = torch.full((batch.hq // 2,), 0.5, device="cuda")
        bias = U.bias_of(batch, 32, 2)[0].cuda()
        for kind in ("diff", "bias"):
            out = U.marked(batch.T, batch.hq // 2, 128) if kind == "diff" else U.marked(batch.T, batch.hq, 64)
            kw = dict(out=out, workspace=ws, options={"decode_ctas": 16} if batch is not mix else None)
            if kind == "diff":
                calls.append(lambda a=args, x=lam, kw=kw: ops.paged_attention_diff(*a, x, **kw))
            else:
                calls.append(lambda a=args, x=bias, kw=kw: ops.paged_attention_bias(*a, x, buckets, **kw))
            outs.append(out)
    for call, out in zip(calls, outs):
        call()
        torch.cuda.synchronize()
        wants.append(out.clone())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    rng = np.random.default_rng(64)
    for _ in range(40):
        order = rng.integers(0, len(graphs), size=12).tolist() + [0, 0, 1, 1, 2, 2, 3, 3]
        for out in outs:
            out.fill_(7.0)
        for i in order:
            graphs[i].replay()
            if rng.random() < 0.2:
                calls[int(rng.integers(0, len(calls)))]()
        torch.cuda.synchronize()
        for i in set(order):
            assert torch.equal(outs[i], wants[i]), i
    assert ops.get_device_error() == 0
