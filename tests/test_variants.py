"""The attention variants without a GPU: the oracle against plain loops, the buckets, and every refusal."""

import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import variants as OV
from paged_kv_gqa_14_gb300 import _lib, ops
from paged_kv_gqa_14_gb300 import build as B
from paged_kv_gqa_14_gb300 import workloads as W


@pytest.fixture(scope="module")
def lib():
    B.build()
    return _lib.load()


def _batch():
    bt = W.make_batch([5, 20, 3], [1, 4, 0], 8, 2, 64, 8, seed=3, block_size=8)
    q, kc, vc = oracle.kv_append(bt.q, bt.k, bt.v, bt.positions, bt.slot_mapping, bt.k_cache, bt.v_cache, bt.rope_theta)
    return q, kc, vc, bt.block_tables, bt.context_lens, bt.query_start_loc, 0.125


def _weights(q, keys, scale, bias=None):
    s = [scale * float(q @ k) + (bias[j] if bias is not None else 0.0) for j, k in enumerate(keys)]
    m = max(s)
    if m == -math.inf:
        return [0.0] * len(s)
    e = [math.exp(x - m) for x in s]
    return [x / sum(e) for x in e]


def test_oracle_of_the_bias_against_plain_loops():
    q, kc, vc, bt, ctx, qsl, scale = args = _batch()
    starts = [0, 1, 2, 5, 9]
    bias = np.random.default_rng(0).normal(size=(5, 8))
    bias[1, 3] = -np.inf
    bias[:, 7] = -np.inf
    out, slack = OV.paged_attention_bias(*args, bias, starts)
    assert np.all(slack[~np.isnan(out)] >= 0)
    for b in range(3):
        K, V = oracle.gather_sequence_kv(kc, vc, bt[b], ctx[b])
        n = qsl[b + 1] - qsl[b]
        for r in range(n):
            pos = ctx[b] - n + r
            for h in range(8):
                add = [bias[max(i for i in range(5) if starts[i] <= pos - j), h] for j in range(pos + 1)]
                w = _weights(oracle.bf16_bits_to_f64(q[qsl[b] + r, h]), K[: pos + 1, h // 4], scale, add)
                want = sum(x * v for x, v in zip(w, V[: pos + 1, h // 4]))
                np.testing.assert_allclose(out[qsl[b] + r, h], want, rtol=1e-12, atol=1e-13)
    assert np.all(out[:, 7] == 0)  # every key taken out


@pytest.mark.parametrize("norm", (False, True))
def test_oracle_of_the_difference_against_plain_loops(norm):
    q, kc, vc, bt, ctx, qsl, scale = args = _batch()
    rng = np.random.default_rng(1)
    lam, weight = rng.uniform(size=(5, 4)), rng.normal(size=128) if norm else None
    out, _ = OV.paged_attention_diff(*args, lam, weight, 1e-3, 0.7)
    for b in range(3):
        K, V = oracle.gather_sequence_kv(kc, vc, bt[b], ctx[b])
        n = qsl[b + 1] - qsl[b]
        for r in range(n):
            t, pos = qsl[b] + r, ctx[b] - n + r
            for h in range(4):
                g = 0  # two kv heads are one pair
                w0 = _weights(oracle.bf16_bits_to_f64(q[t, 2 * h]), K[: pos + 1, 2 * g], scale)
                w1 = _weights(oracle.bf16_bits_to_f64(q[t, 2 * h + 1]), K[: pos + 1, 2 * g + 1], scale)
                x = sum((a - lam[t, h] * c) * np.concatenate([v[2 * g], v[2 * g + 1]]) for a, c, v in zip(w0, w1, V))
                if norm:
                    x = weight * x / math.sqrt(float(np.mean(x * x)) + 1e-3)
                np.testing.assert_allclose(out[t, h], 0.7 * x, rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("num_buckets, max_distance", [(2, 2), (3, 5), (8, 8), (32, 128), (32, 256), (64, 64), (64, 2048),
                                                       (128, 2088), (128, 8192), (7, 31)])
def test_log_buckets(lib, num_buckets, max_distance):
    b = ops.relative_buckets(num_buckets, max_distance)
    starts = list(b.starts)[:num_buckets]
    assert b.num_buckets == num_buckets and starts == OV.log_starts(num_buckets, max_distance)
    # the formula in floating point, away from borders
    e = num_buckets // 2
    for n in range(max_distance + 3):
        x = n if n < e else e + math.log(n / e) / math.log(max_distance / e) * (num_buckets - e)
        if abs(x - round(x)) > 1e-9 or n < e:
            assert OV.bucket_of(n, starts) == min(int(x), num_buckets - 1)


def test_log_buckets_on_a_border():
    # log(32 / 16) / log(256 / 16) 16 = 4 exactly: floating point may fall below it
    assert list(ops.relative_buckets(32, 256).starts)[20] == 32


def test_bucket_refusals(lib):
    r = _lib.RelativeBuckets()
    for nb, far, status in ((1, 5, 2), (129, 500, 2), (32, 16, 2), (32, 0, 2), (32, -5, 2), (128, 20000, 5)):
        assert lib.pkv_relative_buckets_log(nb, far, ctypes.byref(r)) == status, (nb, far)
    assert lib.pkv_relative_buckets_log(32, 128, None) == 1
    with pytest.raises(_lib.PkvError, match="PKV_ERR_SHAPE"):
        ops.relative_buckets(32, 10)
    for bad in ([], [1, 2], [0, 3, 2], list(range(129)), [0, 2**31]):
        with pytest.raises(ValueError, match="starts must"):
            ops.relative_buckets(starts=bad)
    with pytest.raises(ValueError, match="not both"):
        ops.relative_buckets(4, starts=[0])
    with pytest.raises(ValueError, match="needs"):
        ops.relative_buckets(4)
    b = ops.relative_buckets(starts=[0, 0, 4])
    assert b.num_buckets == 3 and list(b.starts)[:3] == [0, 0, 4]


def _call(lib, kind, **kw):
    a = dict(q=256, qs=512, qh=64, kc=256, vc=256, nb=8, bs=16, bt=256, bts=4, mb=4, cl=256, qsl=256, B=2, out=256, os=512,
             oh=64 if kind == "bias" else 128, T=2, hq=8, hkv=4, d=64, scale=0.125, ws=256, wsb=1 << 30, stream=None, opt=None,
             table=256, ts=8, is16=0, lam=256, ls=0, w=256, eps=1e-5, f=0.5, starts=(0, 1, 4), size=None)
    a.update(kw)
    head = (a["q"], a["qs"], a["qh"], a["kc"], a["vc"], a["nb"], a["bs"], a["bt"], a["bts"], a["mb"], a["cl"], a["qsl"], a["B"],
            a["out"], a["os"], a["oh"], a["T"], a["hq"], a["hkv"], a["d"], a["scale"])
    tail = (a["ws"], a["wsb"], a["stream"], a["opt"])
    if kind == "diff":
        return lib.pkv_paged_attention_diff(*head, a["lam"], a["ls"], a["w"], a["eps"], a["f"], *tail)
    b = None
    if a["starts"] is not None:
        b = _lib.RelativeBuckets()
        b.struct_size = ctypes.sizeof(b) if a["size"] is None else a["size"]
        b.num_buckets = len(a["starts"])
        for i, s in enumerate(a["starts"][: _lib.MAX_BUCKETS]):
            b.starts[i] = s
        b = ctypes.byref(b)
    return lib.pkv_paged_attention_bias(*head, a["table"], a["ts"], a["is16"], b, *tail)


@pytest.mark.parametrize("kind", ("bias", "diff"))
def test_refusals_of_the_c_entry_points(lib, kind):
    call = lambda **kw: _call(lib, kind, **kw)
    opt = _lib.AttentionOptions()
    opt.struct_size = ctypes.sizeof(opt)
    opt.decode_kernel = 1
    other = _lib.AttentionOptions()
    other.struct_size = ctypes.sizeof(other)
    other.prefill_kernel = 1
    for want, bad in ((0, dict(T=0)), (0, dict(B=0)), (1, dict(q=None)), (1, dict(out=None)), (1, dict(kc=None)),
                      (2, dict(T=-1)), (2, dict(hq=9)), (2, dict(nb=0)), (2, dict(scale=0.0)), (2, dict(scale=-1.0)),
                      (2, dict(scale=math.inf)), (2, dict(scale=math.nan)), (3, dict(bts=3)), (3, dict(qs=-8)), (3, dict(qs=0)), (3, dict(qh=0)),
                      (3, dict(oh=8)), (4, dict(q=264)), (4, dict(qs=516)), (4, dict(out=264)), (5, dict(d=96)),
                      (5, dict(bs=24)), (5, dict(hq=36)), (5, dict(hkv=16, hq=16)),
                      (5, dict(opt=ctypes.byref(opt))), (5, dict(opt=ctypes.byref(other)))):
        assert call(**bad) == want, bad
    mine = {"bias": ((1, dict(starts=None)), (1, dict(table=None)), (2, dict(starts=())), (2, dict(starts=(1, 2))),
                     (2, dict(starts=(0, 5, 4))), (2, dict(size=12)), (2, dict(is16=2)), (3, dict(ts=7)),
                     (4, dict(table=258)), (4, dict(table=257, is16=1)), (5, dict(starts=(0, 8193)))),
            "diff": ((1, dict(lam=None)), (2, dict(eps=-1.0)), (2, dict(eps=math.nan)), (2, dict(f=math.inf)),
                     (3, dict(ls=-4)), (4, dict(lam=258)), (4, dict(w=264)), (5, dict(hkv=1, hq=8)))}
    for want, bad in mine[kind]:
        assert call(**bad) == want, bad


def test_workspace_of_the_difference(lib):
    size = lib.pkv_paged_attention_diff_workspace_size
    for bad in ((-1, 1, 8, 4, 64, 4, 7), (1, 1, 8, 4, 96, 4, 7), (1, 1, 7, 1, 64, 4, 7), (1, 1, 9, 3, 64, 4, 7),
                (1, 1, 8, 4, 64, 4, -1), (1, 1, 8, 4, 64, -1, 7), (1, 1, 10, 4, 64, 4, 7)):
        assert size(*bad) == 0, bad
    plain = lib.pkv_paged_attention_workspace_size_ex(4, 4, 8, 4, 64, 4, 7)
    assert size(4, 4, 8, 4, 64, 4, 7) >= plain > 0


def _tensors():
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    pool = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    idx = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32), torch.arange(3, dtype=torch.int32)
    return q, pool, pool, *idx


def test_calls_name_what_is_wrong(lib):
    call = _tensors()
    b = ops.relative_buckets(8, 16)
    bias, lam, ws = torch.zeros(8, 4), torch.zeros(2), torch.zeros(1 << 16, dtype=torch.uint8)
    out = torch.empty(2, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="buckets must come from relative_buckets"):
        ops.paged_attention_bias(*call, 0.1, bias, 8)
    with pytest.raises(TypeError, match="scale must be a number"):
        ops.paged_attention_bias(*call, "big", bias, b, out=torch.empty_like(call[0]), workspace=ws)
    with pytest.raises(TypeError, match="norm_eps must be a number"):
        ops.paged_attention_diff(*call, 0.1, lam, norm_eps=None, out=out, workspace=ws)
    with pytest.raises(TypeError, match="max_blocks_per_seq must be an integer"):
        ops.paged_attention_diff(*call, 0.1, lam, max_blocks_per_seq=1.5, out=out, workspace=ws)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        ops.paged_attention_diff(*call, 0.1, lam, out=out, workspace=ws)
    with pytest.raises(TypeError, match="q must be a torch.Tensor"):
        ops.paged_attention_bias(None, *call[1:], 0.1, bias, b)
