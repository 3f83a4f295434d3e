"""paged_attention_bias and paged_attention_diff against the 64-bit oracle."""

import numpy as np
import pytest
import torch

import oracle
from oracle import variants as OV
from paged_kv_gqa_14_gb300 import ops
from paged_kv_gqa_14_gb300 import workloads as W
from tests import variants_util as U
from tests.gpu_util import bf16_to_dev, idx_to_dev

pytestmark = pytest.mark.gpu

HEADS_DIFF = [(2, 2), (4, 4), (6, 2), (16, 8), (14, 2), (32, 4), (24, 8), (64, 8), (20, 4)]  # (Hq, Hkv)
HEADS_BIAS = HEADS_DIFF + [(1, 1), (7, 1), (8, 1), (3, 1)]
T5 = (32, 128)


def both(batch, seed=0, what="", norm=True, buckets=T5, bf16=False, **kw):
    """The two operators on one batch."""
    if batch.hkv % 2 == 0:
        U.check_diff(batch, U.lam_of(batch, seed, per_token=seed % 2 == 1), U.weight_of(batch, seed) if norm else None,
                     out_scale=0.5, what=what + " diff", **kw)
    b = ops.relative_buckets(*buckets)
    bias, bias64 = U.bias_of(batch, buckets[0], seed, bf16)
    U.check_bias(batch, b, bias, bias64, OV.log_starts(*buckets), what=what + " bias", **kw)


# ------------------------------------------------------------------ decode
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("hq, hkv", HEADS_BIAS)
def test_decode_heads(hq, hkv, d):
    ctx = [1, 2, 15, 16, 17, 33, 100, 129, 300]
    both(U.Batch(ctx, [1] * len(ctx), hq, hkv, d, seed=hq + hkv), seed=hq, norm=hq % 3 != 0)


@pytest.mark.parametrize("bs", (8, 16, 32, 64, 128))
@pytest.mark.parametrize("d, hq, hkv", [(64, 4, 2), (128, 8, 4), (128, 16, 8), (64, 8, 8)])
def test_decode_block_sizes(bs, d, hq, hkv):
    ctx = [1, 7, 8, 9, 63, 64, 65, 128, 129, 200, 257, 1000]
    both(U.Batch(ctx, [1] * len(ctx), hq, hkv, d, bs=bs, seed=bs), seed=1)


@pytest.mark.parametrize("ctas", (1, 2, 3, 7, 40))
def test_decode_grids(ctas):
    # entries cut into few and many pieces, several entries to a CTA
    ctx = [700, 3, 40, 1, 1500, 90]
    b = U.Batch(ctx, [1] * len(ctx), 8, 2, 64, seed=ctas)
    both(b, options={"decode_ctas": ctas})
    both(U.Batch([2000], [1], 16, 8, 128, seed=ctas + 9), options={"decode_ctas": ctas})


def test_decode_of_many_sequences():
    rng = np.random.default_rng(5)
    both(U.Batch(rng.integers(1, 120, size=700), [1] * 700, 4, 2, 64, seed=6))


def test_decode_long_context_in_pieces():
    both(U.Batch([9000], [1], 8, 4, 128, bs=64, seed=3))
    both(U.Batch([5003, 1, 4097], [1, 1, 1], 4, 2, 64, seed=4))


def test_idle_sequences_and_rows_behind_the_last():
    both(U.Batch([50, 20, 300, 8], [1, 0, 1, 0], 8, 2, 64, seed=1, extra_tokens=3))
    both(U.Batch([50, 20, 300], [0, 0, 40], 8, 2, 64, seed=1, extra_tokens=5))


def test_longer_spans_among_empty_ones():
    # no more tokens than sequences: every row of the span is a decode entry
    both(U.Batch([90, 5, 6, 7, 30], [4, 0, 0, 0, 1], 8, 4, 128, seed=2))


# ------------------------------------------------------------------ prefill
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("hq, hkv", HEADS_BIAS)
def test_prefill_heads(hq, hkv, d):
    both(U.Batch([70, 190, 2, 140], [70, 60, 2, 3], hq, hkv, d, seed=hq * 3 + hkv), seed=hq + 1, norm=hq % 3 != 0)


@pytest.mark.parametrize("bs", (8, 16, 32, 64, 128))
@pytest.mark.parametrize("d, hq, hkv", [(64, 4, 2), (128, 8, 4), (128, 4, 4)])
def test_prefill_block_sizes(bs, d, hq, hkv):
    both(U.Batch([127, 128, 129, 300, 513], [127, 2, 129, 33, 64], hq, hkv, d, bs=bs, seed=bs + d))


@pytest.mark.parametrize("n", (2, 3, 17, 18, 19, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257))
def test_prefill_span_lengths(n):
    # rows that end inside a tile, keys that end inside a page
    both(U.Batch([n, n + 128, n + 77], [n] * 3, 14, 2, 64, seed=n), seed=n)
    both(U.Batch([n + 255], [n], 4, 2, 128, seed=n), seed=n)


def test_prefill_many_items_to_a_cta():
    ctx = np.random.default_rng(8).integers(40, 700, size=30)
    both(U.Batch(ctx, np.minimum(ctx, 38), 16, 8, 64, seed=9))


def test_long_prefill():
    both(U.Batch([3300], [300], 4, 2, 128, bs=32, seed=10))
    both(U.Batch([2500], [1500], 2, 2, 64, seed=11))


def test_mixed_batches():
    ctx = [300, 1, 45, 700, 260, 64, 1200]
    for options in (None, {"overlap": False}, {"plan_early": True}):
        both(U.Batch(ctx, [1, 1, 45, 1, 130, 2, 1], 16, 8, 128, seed=12), options=options)
    both(U.Batch(ctx, [1, 1, 45, 1, 130, 2, 1], 14, 2, 64, bs=8, seed=13))


# ------------------------------------------------------------------ the bias
@pytest.mark.parametrize("buckets", [(2, 3), (8, 9), (64, 2048), (128, 1000), (32, 8000)])
@pytest.mark.parametrize("bf16", (False, True))
def test_bucket_counts(buckets, bf16):
    both(U.Batch([2300, 700, 129, 3], [1, 1, 129, 2], 4, 1, 64, seed=14), buckets=buckets, bf16=bf16)
    both(U.Batch([1100], [1], 4, 2, 128, seed=15), buckets=buckets, bf16=bf16)


def _custom(batch, starts, bias, what=""):
    b = ops.relative_buckets(starts=starts)
    return U.check_bias(batch, b, torch.from_numpy(bias), bias.astype(np.float64), starts, what=what)


@pytest.mark.parametrize("starts", [[0], [0, 0, 5, 5, 5, 9], [0, 1], [0, 8192], list(range(0, 1280, 10))])
def test_any_starts(starts):
    for ctx, n in (([9000, 130, 1], [1, 1, 1]), ([300, 4000], [300, 20])):
        batch = U.Batch(ctx, n, 4, 2, 64, seed=16)
        _custom(batch, starts, np.random.default_rng(1).normal(size=(len(starts), 4)).astype(np.float32))


def test_a_window_and_rows_without_keys():
    # -inf in the last bucket: a window of 40 keys; in the first: the own key taken out, so the first row has none
    rng = np.random.default_rng(2)
    for ctx, n in (([500, 41, 40, 1, 2], [1] * 5), ([300, 60], [300, 60]), ([700, 1], [130, 1])):
        for hq, hkv, d in ((4, 2, 64), (7, 1, 128)):
            batch = U.Batch(ctx, n, hq, hkv, d, seed=17)
            for row in (-1, 0):
                bias = rng.normal(size=(3, hq)).astype(np.float32)
                bias[row] = -np.inf
                _custom(batch, [0, 20, 40], bias)
            bias[:] = -np.inf
            assert _custom(batch, [0, 20, 40], bias) == 0.0  # nothing left: zeros


@pytest.mark.parametrize("low", (-3.4028234663852886e38, -1e30, -3.0e4, 1e30))
def test_biases_that_swallow_the_scores(low):
    # keys that share such a bias are weighted alike where it is all there is, and not at all beside others (above them
    # where it is large and positive)
    bias = np.zeros((3, 4), np.float32)
    bias[2] = low
    for ctx, n in (([500, 41, 1], [1, 1, 1]), ([300], [300])):
        batch = U.Batch(ctx, n, 4, 2, 64, seed=18)
        _custom(batch, [0, 20, 40], bias)
        if abs(low) > 1e20:
            _custom(batch, [0, 20, 40], np.full_like(bias, low))


def test_bias_of_infinity_and_nan_stay_in_their_rows():
    batch = U.Batch([100, 10], [1, 1], 4, 2, 64, seed=19)
    bias = np.zeros((3, 4), np.float32)
    bias[2, 1] = np.nan
    bias[2, 2] = np.inf
    b = ops.relative_buckets(starts=[0, 20, 40])
    out = ops.paged_attention_bias(*batch.dev(), torch.from_numpy(bias).cuda(), b)
    assert torch.isnan(out[0, 1:3]).all() and torch.isfinite(out[0, 0]).all() and torch.isfinite(out[0, 3]).all()
    assert torch.isfinite(out[1]).all()  # ten keys: the last bucket is not met


def test_bias_rows_of_a_wider_table():
    batch = U.Batch([300, 130], [1, 130], 4, 2, 64, seed=20)
    wide = torch.randn(32, 9, generator=torch.Generator().manual_seed(1))
    b = ops.relative_buckets(*T5)
    ref, slack = OV.paged_attention_bias(*batch.host(), wide[:, 3:7].double().numpy(), OV.log_starts(*T5))
    out = U.marked(batch.T, 4, 64)
    ops.paged_attention_bias(*batch.dev(), wide.cuda()[:, 3:7], b, out=out)
    U.within(out, ref, slack)


# ------------------------------------------------------------------ values and layouts
@pytest.mark.parametrize("gain", (8.0, 100.0, 3.0e4))
def test_large_scores(gain):
    both(U.Batch([400, 1, 129], [1, 1, 129], 8, 2, 64, seed=21, gain=gain), norm=False)


def test_equal_maps_leave_one_minus_lambda():
    # one key: both maps are 1, x = (1 - lam) v, whatever the scores
    batch = U.Batch([1, 1, 1], [1, 1, 1], 4, 2, 64, seed=22, gain=100.0)
    lam = np.array([0.25, 1.0], np.float32)
    out = ops.paged_attention_diff(*batch.dev(), torch.from_numpy(lam).cuda())
    ref, _ = OV.paged_attention_diff(*batch.host(), lam)
    assert torch.equal(out.cpu(), torch.from_numpy(ref).to(torch.bfloat16))
    # and with the norm a head whose maps cancel is 0, not infinite
    out = ops.paged_attention_diff(*batch.dev(), torch.from_numpy(lam).cuda(), norm_weight=torch.ones(128, device="cuda"))
    assert torch.isfinite(out).all() and (out[:, 1] == 0).all()


def test_strides_of_q_out_lam_and_tables():
    batch = U.Batch([300, 77, 130], [1, 1, 130], 8, 4, 64, seed=23)
    q, kc, vc, bt, ctx, qsl, scale = batch.dev()
    T = batch.T
    packed = torch.zeros(T, 8 + 5, 72, dtype=torch.bfloat16, device="cuda")
    packed[:, 2:10, :64] = q
    wide = torch.full((bt.shape[0], bt.shape[1] + 3), -1, dtype=torch.int32, device="cuda")
    wide[:, :bt.shape[1]] = bt
    lam = U.lam_of(batch, 1, True)
    lam_wide = torch.zeros(T, 7, device="cuda")
    lam_wide[:, 2:6] = torch.from_numpy(lam)
    ref, slack = OV.paged_attention_diff(*batch.host(), lam, None)
    out = U.marked(T, 6, 144)
    got = ops.paged_attention_diff(packed[:, 2:10, :64], kc, vc, wide, ctx, qsl, scale, lam_wide[:, 2:6],
                                   out=out[:, 1:5, 8:136], max_blocks_per_seq=bt.shape[1])
    U.within(got, ref, slack)
    rest = out.clone()
    rest[:, 1:5, 8:136] = 7.0
    assert (rest == 7.0).all()
    b = ops.relative_buckets(*T5)
    bias, bias64 = U.bias_of(batch, 32, 2)
    ref, slack = OV.paged_attention_bias(*batch.host(), bias64, OV.log_starts(*T5))
    out = U.marked(8, T, 64).transpose(0, 1)  # head-major
    U.within(ops.paged_attention_bias(packed[:, 2:10, :64], kc, vc, wide, ctx, qsl, scale, bias.cuda(), b, out=out), ref,
             slack)


def test_without_an_output_and_nothing_to_do():
    batch = U.Batch([30, 20], [1, 20], 4, 2, 64, seed=24)
    q, kc, vc, bt, ctx, qsl, scale = batch.dev()
    lam, b, bias = torch.ones(2, device="cuda"), ops.relative_buckets(*T5), torch.zeros(32, 4, device="cuda")
    assert ops.paged_attention_diff(q, kc, vc, bt, ctx, qsl, scale, lam).shape == (21, 2, 128)
    assert ops.paged_attention_bias(q, kc, vc, bt, ctx, qsl, scale, bias, b).shape == (21, 4, 64)
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert ops.paged_attention_diff(q[:0], kc, vc, bt, ctx, none, scale, lam).shape == (0, 2, 128)
    assert ops.paged_attention_bias(q[:0], kc, vc, bt, ctx, none, scale, bias, b).shape == (0, 4, 64)


def test_a_bias_of_zero_is_plain_attention():
    batch = U.Batch([300, 77, 130], [1, 1, 130], 8, 4, 64, seed=25)
    ref = oracle.paged_attention(*batch.host())
    b = ops.relative_buckets(*T5)
    _, slack = OV.paged_attention_bias(*batch.host(), np.zeros((32, 8)), OV.log_starts(*T5))
    out = U.marked(batch.T, 8, 64)
    U.within(ops.paged_attention_bias(*batch.dev(), torch.zeros(32, 8, device="cuda"), b, out=out), ref, slack)


# ------------------------------------------------------------------ as they are used
def test_a_step_of_append_and_difference():
    """Two layers' steps: kv_append rotates and writes, the attention follows with early planning and streaming."""
    for opts in (None, ops.attention_options({"plan_early": True, "stream_early": True})):
        for ctx, spans in (([700, 33, 1, 160], [1, 1, 1, 1]), ([700, 33, 90, 160], [1, 1, 90, 7])):
            bt = W.make_batch(ctx, spans, 16, 8, 128, 80, seed=26)
            dq, k, v = bf16_to_dev(bt.q), bf16_to_dev(bt.k), bf16_to_dev(bt.v)
            kc, vc = bf16_to_dev(bt.k_cache), bf16_to_dev(bt.v_cache)
            idx = [idx_to_dev(x) for x in (bt.block_tables, bt.context_lens, bt.query_start_loc)]
            lam = torch.full((8,), 0.5, device="cuda")
            ws = ops.alloc_workspace(bt.num_tokens, 4, 16, 8, 128, bt.block_tables.shape[1], diff=True)
            out = U.marked(bt.num_tokens, 8, 256)
            for _ in range(2):  # the second on a workspace and a cache that were used
                q = dq.clone()
                torch.cuda.synchronize()
                ops.kv_append(q, k, v, idx_to_dev(bt.positions), idx_to_dev(bt.slot_mapping), kc, vc, bt.rope_theta)
                ops.paged_attention_diff(q, kc, vc, *idx, bt.scale, lam, out=out, workspace=ws, options=opts)
            torch.cuda.synchronize()
            assert ops.get_device_error() == 0
            qr, okc, ovc = oracle.kv_append(bt.q, bt.k, bt.v, bt.positions, bt.slot_mapping, bt.k_cache, bt.v_cache,
                                            bt.rope_theta)
            # (the kernel's q and k may round the other way next to a border: the reference takes them as they are)
            qr, okc = (x.contiguous().view(torch.int16).cpu().numpy().view(np.uint16) for x in (q, kc))
            ref, slack = OV.paged_attention_diff(qr, okc, ovc, bt.block_tables, bt.context_lens, bt.query_start_loc,
                                                 bt.scale, np.full(8, 0.5))
            U.within(out, ref, slack)


def test_a_step_without_rotation_and_the_bias():
    """A model with a relative bias has no rotation: the append's positions are 0."""
    bt = W.make_batch([200, 50, 70], [1, 1, 70], 8, 2, 64, 40, seed=27)
    q, k, v = bf16_to_dev(bt.q), bf16_to_dev(bt.k), bf16_to_dev(bt.v)
    kc, vc = bf16_to_dev(bt.k_cache), bf16_to_dev(bt.v_cache)
    idx = [idx_to_dev(x) for x in (bt.block_tables, bt.context_lens, bt.query_start_loc)]
    zero = torch.zeros(bt.num_tokens, dtype=torch.int64, device="cuda")
    ops.kv_append(q, k, v, zero, idx_to_dev(bt.slot_mapping), kc, vc, 1e4)
    assert torch.equal(q, bf16_to_dev(bt.q))
    b = ops.relative_buckets(*T5)
    bias = torch.randn(32, 8, generator=torch.Generator().manual_seed(3))
    out = U.marked(bt.num_tokens, 8, 64)
    ops.paged_attention_bias(q, kc, vc, *idx, 1.0, bias.cuda(), b, out=out)
    kc_, vc_ = bt.k_cache.copy(), bt.v_cache.copy()
    bs = bt.block_size
    for t, s in enumerate(bt.slot_mapping):
        kc_[s // bs, s % bs], vc_[s // bs, s % bs] = bt.k[t], bt.v[t]
    ref, slack = OV.paged_attention_bias(bt.q, kc_, vc_, bt.block_tables, bt.context_lens, bt.query_start_loc, 1.0,
                                         bias.double().numpy(), OV.log_starts(*T5))
    U.within(out, ref, slack)


def test_the_same_bits_again_and_on_another_stream():
    batch = U.Batch([1500, 3, 400, 90], [1, 1, 200, 1], 16, 8, 64, seed=28)
    args, lam = batch.dev(), torch.from_numpy(U.lam_of(batch, 1)).cuda()
    bias, b = U.bias_of(batch, 32, 2)[0].cuda(), ops.relative_buckets(*T5)
    first = ops.paged_attention_diff(*args, lam), ops.paged_attention_bias(*args, bias, b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):
        for stream in (None, side):
            again = ops.paged_attention_diff(*args, lam, stream=stream), ops.paged_attention_bias(*args, bias, b, stream=stream)
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_two_calls_at_once():
    one = U.Batch([1500, 300], [1, 1], 16, 8, 64, seed=29)
    two = U.Batch([900, 64, 130], [1, 1, 130], 8, 2, 64, seed=30)
    lam, bias = torch.from_numpy(U.lam_of(one, 1)).cuda(), U.bias_of(two, 32, 2)[0].cuda()
    b = ops.relative_buckets(*T5)
    a1, a2 = one.dev(), two.dev()
    want = ops.paged_attention_diff(*a1, lam), ops.paged_attention_bias(*a2, bias, b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(30):
        got.append((ops.paged_attention_diff(*a1, lam, stream=s1), ops.paged_attention_bias(*a2, bias, b, stream=s2)))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for g in got for x, y in zip(g, want))


def test_captured_calls_that_share_a_workspace():
    dec = U.Batch([300, 77, 1200], [1, 1, 1], 8, 2, 64, seed=31)
    mix = U.Batch([300, 77, 200], [1, 77, 60], 8, 2, 64, seed=32)
    T = max(dec.T, mix.T)
    ws = ops.alloc_workspace(T, 3, 8, 2, 64, 128, diff=True)
    b = ops.relative_buckets(*T5)
    calls, graphs, outs, wants = [], [], [], []
    for batch in (dec, mix):
        args, lam, bias = batch.dev(), torch.from_numpy(U.lam_of(batch, 1)).cuda(), U.bias_of(batch, 32, 2)[0].cuda()
        calls.append(lambda out, a=args, x=lam: ops.paged_attention_diff(*a, x, out=out, workspace=ws))
        outs.append(U.marked(batch.T, 4, 128))
        calls.append(lambda out, a=args, x=bias: ops.paged_attention_bias(*a, x, b, out=out, workspace=ws))
        outs.append(U.marked(batch.T, 8, 64))
    for call, out in zip(calls, outs):
        call(out)
        torch.cuda.synchronize()
        wants.append(out.clone())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(out)
        graphs.append(g)
    for order in ((0, 1, 2, 3), (3, 1, 2, 0), (2, 2, 0, 0)):
        for out in outs:
            out.fill_(7.0)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in order:
            assert torch.equal(outs[i], wants[i])
    assert ops.get_device_error() == 0


def test_captured_steps_with_shared_items_follow_their_inputs():
    # the spans and lengths are read in each replay: few long items, then many short ones, then none
    batches = [U.Batch([2500, 1100, 7], [12, 3, 1], 8, 4, 64, seed=51), U.Batch([9, 8, 20], [8, 3, 5], 8, 4, 64, seed=52),
               U.Batch([2000, 16, 1], [14, 1, 1], 8, 4, 64, seed=53)]
    T = 16
    assert all(b.T == T for b in batches)
    width = max(b.bt.block_tables.shape[1] for b in batches)
    pool = max(b.kc.shape[0] for b in batches)
    q, kc, vc = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((T, 8, 64), (pool, 16, 4, 64), (pool, 16, 4, 64)))
    bt, ctx, qsl = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((3, width), (3,), (4,)))
    ctx.fill_(6)
    qsl.copy_(torch.tensor([0, 6, 11, 16]))
    bias, bias64 = U.bias_of(batches[0], 32, 2)
    lam, bias, b = torch.full((4,), 0.4, device="cuda"), bias.cuda(), ops.relative_buckets(*T5)
    ws = ops.alloc_workspace(T, 3, 8, 4, 64, width, diff=True)
    outs = U.marked(T, 4, 128), U.marked(T, 8, 64)
    args = (q, kc, vc, bt, ctx, qsl, 64**-0.5)

    def step():
        ops.paged_attention_diff(*args, lam, out=outs[0], workspace=ws)
        ops.paged_attention_bias(*args, bias, b, out=outs[1], workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (0, 1, 2, 0):
        x = batches[i].dev()
        q.copy_(x[0])
        kc[:x[1].shape[0]].copy_(x[1])
        vc[:x[2].shape[0]].copy_(x[2])
        bt[:, :x[3].shape[1]].copy_(x[3])
        ctx.copy_(x[4])
        qsl.copy_(x[5])
        graph.replay()
        torch.cuda.synchronize()
        U.within(outs[0], *OV.paged_attention_diff(*batches[i].host(), np.full(4, np.float32(0.4))), what=f"diff {i}")
        U.within(outs[1], *OV.paged_attention_bias(*batches[i].host(), bias64, OV.log_starts(*T5)), what=f"bias {i}")
    assert ops.get_device_error() == 0


# ------------------------------------------------------------------ what may be wrong with a call
def test_bad_tables_are_flagged():
    b, bias = ops.relative_buckets(*T5), torch.zeros(32, 8, device="cuda")
    for spans in ([1, 1, 1, 1], [1, 40, 1, 1]):
        batch = U.Batch([100, 60, 30, 10], spans, 8, 2, 64, seed=33)
        q, kc, vc, bt, ctx, qsl, scale = batch.dev()
        lam = torch.ones(4, device="cuda")
        for call in (lambda *a: ops.paged_attention_diff(*a, lam), lambda *a: ops.paged_attention_bias(*a, bias, b)):
            good = call(q, kc, vc, bt, ctx, qsl, scale)
            assert ops.get_device_error() == 0

            def only(bad_rows, got):
                keep = torch.ones(batch.T, dtype=torch.bool)
                keep[bad_rows] = False
                assert torch.equal(got[keep.cuda()], good[keep.cuda()])

            for bad_id in (-1, 10**6):
                t = bt.clone()
                t[2, 1] = bad_id
                got = call(q, kc, vc, t, ctx, qsl, scale)
                assert ops.get_device_error() == 0x2
                only(slice(int(qsl[2]), int(qsl[3])), got)
            c = ctx.clone()
            c[0] = bt.shape[1] * 16 + 1
            call(q, kc, vc, bt, c, qsl, scale)
            assert ops.get_device_error() == 0x8
            c[0] = 2**31 - 1
            call(q, kc, vc, bt, c, qsl, scale)
            assert ops.get_device_error() == 0x8
            c = ctx.clone()
            c[3] = 0
            call(q, kc, vc, bt, c, qsl, scale)
            assert ops.get_device_error() == 0x4
            s = qsl.clone()
            s[3] = 0  # goes back
            call(q, kc, vc, bt, ctx, s, scale)
            assert ops.get_device_error() & 0x4
            s = qsl.clone()
            s[4] = batch.T + 5
            call(q, kc, vc, bt, ctx, s, scale)
            assert ops.get_device_error() == 0x4
            assert torch.equal(call(q, kc, vc, bt, ctx, qsl, scale), good)


def test_refusals():
    batch = U.Batch([100, 60], [1, 1], 8, 2, 64, seed=34)
    q, kc, vc, bt, ctx, qsl, scale = args = batch.dev()
    b, bias, lam = ops.relative_buckets(*T5), torch.zeros(32, 8, device="cuda"), torch.ones(4, device="cuda")
    ws = ops.alloc_workspace(2, 2, 8, 2, 64, bt.shape[1], diff=True)
    diff, add = ops.paged_attention_diff, ops.paged_attention_bias
    for error, match, call in (
            (TypeError, "k_cache must be torch.bfloat16", lambda: diff(q, kc.float(), vc, *args[3:], lam)),
            (TypeError, "lam must be one of", lambda: diff(*args, lam.double())),
            (ValueError, r"lam must be \(4,\) or \(2, 4\)", lambda: diff(*args, torch.ones(8, device="cuda"))),
            (ValueError, "norm_weight must be", lambda: diff(*args, lam, norm_weight=torch.ones(64, device="cuda"))),
            (ValueError, "lam must be a CUDA tensor", lambda: diff(*args, lam.cpu())),
            (ValueError, r"out must be \(2, 4, 128\)", lambda: diff(*args, lam, out=torch.empty_like(q))),
            (ValueError, "even number of heads", lambda: diff(q[:, :7], *args[1:], lam)),
            (ValueError, r"bias must be \(32, 8\)", lambda: add(*args, bias[:, :7], b)),
            (TypeError, "bias must be one of", lambda: add(*args, bias.half(), b)),
            (ValueError, "last dim must be contiguous", lambda: add(*args, bias.repeat(1, 2)[:, ::2], b)),
            (ValueError, "more than block_tables' columns", lambda: add(*args, bias, b, max_blocks_per_seq=bt.shape[1] + 1)),
            (ValueError, "num_seqs . 1 entries", lambda: add(q, kc, vc, bt, ctx, qsl[:2], scale, bias, b)),
            (ValueError, "workspace must be", lambda: diff(*args, lam, workspace=ws.cpu())),
            (ops._lib.PkvError, "PKV_ERR_WORKSPACE", lambda: diff(*args, lam, workspace=ws[:512])),
            (ops._lib.PkvError, "PKV_ERR_WORKSPACE", lambda: add(*args, bias, b, workspace=ws[1:])),
            (ops._lib.PkvError, "PKV_ERR_UNSUPPORTED", lambda: add(*args, bias, b, options={"decode_kernel": "simt"})),
            (ops._lib.PkvError, "PKV_ERR_UNSUPPORTED", lambda: diff(*args, lam, options={"prefill_kernel": "mma"})),
            (ops._lib.PkvError, "PKV_ERR_SHAPE", lambda: diff(q, kc, vc, bt, ctx, qsl, -scale, lam)),
            (ops._lib.PkvError, "PKV_ERR_UNSUPPORTED",
             lambda: add(*args, torch.zeros(2, 8, device="cuda"), ops.relative_buckets(starts=[0, 9000])))):
        with pytest.raises(error, match=match):
            call()
    assert ops.get_device_error() == 0
    diff(*args, lam, workspace=ws)
    add(*args, bias, b, workspace=ws)


@pytest.mark.parametrize("hkv, spans, ctx", [(2, [60, 1], 300), (8, [250] * 12 + [1], 300), (2, [60, 1], 2000)])
def test_prefill_waits_run_out_and_report(hkv, spans, ctx):
    """The loaders issue nothing: every other role's wait runs out (about a second, once for a CTA), the CTAs of a cluster
    meet at their barriers all the same (with 2000 keys four pairs share an item), the error is reported and the next call runs as ever."""
    batch = U.Batch([ctx] * len(spans), spans, 2 * hkv, hkv, 64, seed=35)
    args, lam = batch.dev(), torch.from_numpy(U.lam_of(batch, 1)).cuda()
    bias, b = U.bias_of(batch, 32, 2)[0].cuda(), ops.relative_buckets(*T5)
    for call in (lambda: ops.paged_attention_diff(*args, lam), lambda: ops.paged_attention_bias(*args, bias, b)):
        want = call()
        ops.set_fault_injection("prefill_no_copies")
        try:
            got = call()
            assert ops.get_device_error() == 0x10
        finally:
            ops.set_fault_injection(None)
        assert torch.equal(got[-1], want[-1])  # the decode row
        assert torch.equal(call(), want)


def test_decode_waits_run_out_and_report():
    batch = U.Batch([300, 40], [1, 1], 4, 2, 64, seed=36)
    args, lam = batch.dev(), torch.from_numpy(U.lam_of(batch, 1)).cuda()
    bias, b = U.bias_of(batch, 32, 2)[0].cuda(), ops.relative_buckets(*T5)
    for call in (lambda: ops.paged_attention_diff(*args, lam), lambda: ops.paged_attention_bias(*args, bias, b)):
        want = call()
        ops.set_fault_injection("decode_no_copies")
        try:
            call()
            assert ops.get_device_error() == 0x10
        finally:
            ops.set_fault_injection(None)
        assert torch.equal(call(), want)


# ------------------------------------------------------------------ items shared by several pairs of CTAs
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("ctx, spans", [
    ([3000], [12]), ([130], [5]), ([129], [129]), ([513], [3]), ([2000, 700, 40], [9, 2, 33]), ([700, 1, 900], [12, 1, 7]),
    ([900] * 5, [2] * 5), ([1100, 500], [70, 60])])
def test_short_spans_behind_long_contexts(ctx, spans, d):
    # keys of an item cut into up to four ranges, some of them empty, beside decodes or not
    for hq, hkv in ((12, 4), (4, 2), (14, 2)):
        both(U.Batch(ctx, spans, hq, hkv, d, seed=hq + len(ctx)), seed=len(ctx), norm=hq != 4)
    both(U.Batch(ctx, spans, 7, 1, d, bs=64, seed=3), seed=1, bf16=True)


def test_short_spans_repeat_bit_for_bit():
    batch = U.Batch([2500, 1800], [12, 30], 24, 4, 64, seed=41)
    args, lam = batch.dev(), torch.from_numpy(U.lam_of(batch, 1)).cuda()
    want = ops.paged_attention_diff(*args, lam)
    for _ in range(20):
        assert torch.equal(ops.paged_attention_diff(*args, lam), want)


# ------------------------------------------------------------------ large pools and batches
@pytest.mark.parametrize("ctx, spans", [([500, 70, 33], [1, 1, 1]), ([500, 70, 33], [1, 70, 1]), ([1500, 1200, 33], [9, 1, 2])])
def test_blocks_past_2_to_the_31_elements(ctx, spans):
    """The same rows in blocks at the end of a pool of 4.4 billion elements (8.8 GB each)."""
    batch = U.Batch(ctx, spans, 16, 8, 128, seed=37)
    q, kc, vc, bt, ctx, qsl, scale = batch.dev()
    lam = torch.from_numpy(U.lam_of(batch, 1)).cuda()
    bias, b = U.bias_of(batch, 32, 2)[0].cuda(), ops.relative_buckets(*T5)
    nb = 270000
    big = [torch.empty(nb, 16, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    for x, small in zip(big, (kc, vc)):
        x[-small.shape[0]:] = small
    far = torch.where(bt >= 0, bt + (nb - kc.shape[0]), bt)
    assert int(far.max()) * 16 * 8 * 128 > 2**32
    for call in (lambda k, v, t: ops.paged_attention_diff(q, k, v, t, ctx, qsl, scale, lam),
                 lambda k, v, t: ops.paged_attention_bias(q, k, v, t, ctx, qsl, scale, bias, b)):
        assert torch.equal(call(*big, far), call(kc, vc, bt))
    assert ops.get_device_error() == 0


def test_mixed_batch_of_more_sequences_than_the_small_planner_takes():
    rng = np.random.default_rng(38)
    ctx = rng.integers(1, 60, size=1100)
    spans = np.ones(1100, int)
    ctx[700], spans[700] = 150, 130
    ctx[20], spans[20] = 40, 40
    both(U.Batch(ctx, spans, 4, 2, 64, seed=39))


@pytest.mark.parametrize("seed", range(6))
def test_random_batches(seed):
    """Sizes, heads, blocks and spans drawn at random, idle sequences among them."""
    rng = np.random.default_rng(1000 + seed)
    hkv = int(rng.choice([2, 4, 8]))
    hq, d, bs = hkv * int(rng.integers(1, 9)), int(rng.choice([64, 128])), int(rng.choice([8, 16, 32, 64, 128]))
    n = int(rng.integers(1, 12))
    ctx = np.exp(rng.uniform(0, np.log(1500), n)).astype(int)
    spans = np.array([int(rng.choice([0, 1, 1, rng.integers(0, c + 1)])) for c in ctx])
    spans = np.minimum(spans, 200)
    buckets = int(rng.integers(2, 129))
    both(U.Batch(ctx, spans, hq, hkv, d, bs=bs, seed=seed), seed=seed, norm=seed % 2 == 0,
         buckets=(buckets, buckets // 2 + int(rng.integers(1, 1500))), bf16=seed % 3 == 0)
