"""The 8-bit cache without a GPU: the oracle's format against torch's casts and closed forms, and the
host-side refusals of the library and the binding."""

import numpy as np
import pytest
import torch

from oracle import q8 as OQ
from oracle import bf16_bits_to_f64, kv_append, positions_and_slots
from paged_kv_gqa_14_gb300 import _lib, ops
from paged_kv_gqa_14_gb300 import build as B
from paged_kv_gqa_14_gb300 import workloads as W

KINDS = ("int8", "e4m3")


@pytest.fixture(scope="module")
def lib():
    B.build()
    return _lib.load()


# ------------------------------------------------------------------------------ the oracle's pins
def test_e4m3_values_are_torch_s():
    codes = torch.arange(256, dtype=torch.int16).to(torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    got = OQ.decode(codes.numpy(), "e4m3")
    assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("kind", KINDS)
def test_every_code_survives_decode_and_encode(kind):
    codes = np.arange(256, dtype=np.uint8)
    if kind == "int8":
        codes = codes[codes != 128]  # -128 is not written
    else:
        codes = codes[(codes & 127) != 127]
    assert np.array_equal(OQ.encode(OQ.decode(codes, kind), kind), codes)


def test_encode_is_torch_s_rounding():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * 2.0 ** rng.integers(-12, 9, 20000), np.arange(-448, 449) / 2.0,
                        np.arange(-64, 65) * 2.0**-11]).astype(np.float32)
    x = np.clip(x, -448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(OQ.encode(x, "e4m3"), want)
    y = np.clip(x, -127, 127)
    want = torch.round(torch.from_numpy(y)).to(torch.int8).numpy().view(np.uint8)
    assert np.array_equal(OQ.encode(y, "int8"), want)


@pytest.mark.parametrize("kind", KINDS)
def test_scale_is_the_smallest_that_fits(kind):
    top = OQ.LARGEST[kind]
    for e in (-100, -99, -3, 0, 7, 60):
        s = 2.0**e
        assert OQ.scale_for(top * s, kind) == s
        assert OQ.scale_for(np.nextafter(top * s, np.inf), kind) == 2 * s
        assert OQ.scale_for(top * s / 2, kind) == max(s / 2, 2.0**-100)
    assert OQ.scale_for(0.0, kind) == 2.0**-100
    x = np.abs(np.random.default_rng(1).standard_normal(1000))
    s = OQ.scale_for(x, kind)
    assert (x <= top * s).all() and (x > top * s / 2).all()


@pytest.mark.parametrize("kind", KINDS)
def test_a_dequantised_value_is_a_bf16_value(kind):
    codes = np.arange(256, dtype=np.uint8)
    codes = codes[(codes & 127) != 127] if kind == "e4m3" else codes
    for e in (-100, -20, 0, 30, 119):
        bits = OQ.dequantise(codes.reshape(1, 1, 1, -1), np.full((1, 1), 2.0**e), kind)
        assert np.array_equal(bf16_bits_to_f64(bits)[0, 0, 0], OQ.decode(codes, kind) * 2.0**e)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bs", (8, 16))
def test_append_stands_within_a_step_of_the_bf16_append(kind, bs):
    """One call with a whole prompt: every value within half a step of what the bf16 cache would hold
    before its own rounding (compared after it: plus half a bf16 step)."""
    bt = W.make_batch([37, 9], [37, 9], 4, 2, 64, 12, seed=3, poison=False, block_size=bs)
    nb = bt.k_cache.shape[0]
    codes = np.zeros(bt.k_cache.shape, np.uint8)
    ones = np.ones((nb, 2))
    q, kc, vc, ks, vs, _ = OQ.kv_append_q8(bt.q, bt.k, bt.v, bt.block_tables, bt.context_lens, bt.query_start_loc,
                                           codes, codes, ones, ones, 1e6, kind)
    pos, slots = positions_and_slots(bt.query_start_loc, bt.context_lens, bt.block_tables, bs, bt.num_tokens)
    q2, k2, v2 = kv_append(bt.q, bt.k, bt.v, pos, slots, np.zeros_like(bt.k_cache), np.zeros_like(bt.v_cache), 1e6)
    assert np.array_equal(q, q2)
    for codes, scale, want in ((kc, ks, k2), (vc, vs, v2)):
        x = bf16_bits_to_f64(want)
        held = OQ.decode(codes, kind)
        step = np.ones_like(held) if kind == "int8" else np.maximum(np.abs(held) / 8, 2.0**-9)
        err = np.abs(held * scale[:, None, :, None] - x)
        written = np.zeros(codes.shape[:2], bool)
        written[slots // bs, slots % bs] = True
        assert (err <= 0.5 * step * scale[:, None, :, None] * 1.0001 + 2.0**-8 * np.abs(x))[written].all()
        assert (err[~written] == 0).all()


@pytest.mark.parametrize("kind", KINDS)
def test_appending_one_by_one_gives_the_same_scales_and_nearly_the_same_values(kind):
    """The scale of a block does not depend on how its tokens came; a value that came early is within
    one step (of the final scale) of what a single call writes."""
    rng = np.random.default_rng(5)
    bs, n, hkv, d = 16, 16, 2, 64
    k = W.normal_bf16(rng, (n, hkv, d))
    v = W.normal_bf16(rng, (n, hkv, d))
    grow = np.ldexp(1.0, np.arange(n) // 3)  # tokens that get larger
    v = OQ.f64_to_bf16_bits(bf16_bits_to_f64(v) * grow[:, None, None])
    table = np.zeros((1, 1), np.int32)
    z, one = np.zeros((1, bs, hkv, d), np.uint8), np.ones((1, hkv))
    whole = OQ.kv_append_q8(k[:, :2], k, v, table, [n], [0, n], z, z, one, one, 1e6, kind)
    kc, vc, ks, vs = z, z, one, one
    for t in range(n):
        _, kc, vc, ks, vs, _ = OQ.kv_append_q8(k[t:t + 1, :2], k[t:t + 1], v[t:t + 1], table, [t + 1], [0, 1], kc, vc, ks,
                                               vs, 1e6, kind)
    assert np.array_equal(ks, whole[3]) and np.array_equal(vs, whole[4])
    a, b = OQ.decode(vc, kind), OQ.decode(whole[2], kind)
    step = np.ones_like(b) if kind == "int8" else np.maximum(np.abs(b) / 8, 2.0**-9)
    assert (np.abs(a - b) <= step).all()


# ------------------------------------------------------------------------------------ refusals
def _append(lib, **kw):
    a = dict(q=16, qs=1024, qh=128, k=16, ks=512, kh=128, v=16, vs=512, vh=128, bt=16, bts=8, mb=8, ctx=16, qsl=16,
             B=2, kc=16, vc=16, sk=16, sv=16, T=4, hq=8, hkv=4, d=128, nb=10, bs=16, fmt=1, theta=1e6)
    a.update(kw)
    return lib.pkv_kv_append_q8(a["q"], a["qs"], a["qh"], a["k"], a["ks"], a["kh"], a["v"], a["vs"], a["vh"], a["bt"],
                                a["bts"], a["mb"], a["ctx"], a["qsl"], a["B"], a["kc"], a["vc"], a["sk"], a["sv"],
                                a["T"], a["hq"], a["hkv"], a["d"], a["nb"], a["bs"], a["fmt"], a["theta"], None)


def test_append_refusals(lib):
    assert _append(lib, d=96) == 5
    for bs in (0, -16, 4, 12, 256):
        assert _append(lib, bs=bs) == 5
    for fmt in (0, 3, -1):
        assert _append(lib, fmt=fmt) == 5
    assert _append(lib, hkv=1025, hq=1025) == 5
    for name in ("q", "k", "v", "bt", "ctx", "qsl", "kc", "vc", "sk", "sv"):
        assert _append(lib, **{name: None}) == 1, name
    for name in ("q", "k", "v", "kc", "vc", "sk", "sv"):
        assert _append(lib, **{name: 8}) == 4, name
    assert _append(lib, nb=1 << 31) == 2
    assert _append(lib, hq=6) == 2
    assert _append(lib, theta=float("nan")) == 2
    assert _append(lib, T=-1) == 2 and _append(lib, B=-1) == 2 and _append(lib, T=(1 << 28) + 1) == 2
    assert _append(lib, bts=4) == 3
    assert _append(lib, qs=1016) == 3
    assert _append(lib, ks=516) == 4
    for bs in (8, 16, 32, 64, 128):
        for fmt in (1, 2):
            assert _append(lib, bs=bs, fmt=fmt, T=0) == 0
    assert _append(lib, B=0) == 0


def _read(lib, **kw):
    a = dict(kc=16, vc=16, sk=16, sv=16, nb=10, bs=16, bt=16, bts=8, mb=8, ctx=16, rsl=16, B=2, ko=16, kos=512, koh=128,
             vo=16, vos=512, voh=128, R=4, hkv=4, d=128, fmt=2)
    a.update(kw)
    return lib.pkv_kv_read_q8(a["kc"], a["vc"], a["sk"], a["sv"], a["nb"], a["bs"], a["bt"], a["bts"], a["mb"], a["ctx"],
                              a["rsl"], a["B"], a["ko"], a["kos"], a["koh"], a["vo"], a["vos"], a["voh"], a["R"],
                              a["hkv"], a["d"], a["fmt"], None)


def test_read_refusals(lib):
    assert _read(lib, d=32) == 5 and _read(lib, bs=24) == 5 and _read(lib, fmt=0) == 5
    for name in ("kc", "vc", "sk", "sv", "bt", "ctx", "rsl", "ko", "vo"):
        assert _read(lib, **{name: None}) == 1, name
    for name in ("kc", "vc", "sk", "sv", "ko", "vo"):
        assert _read(lib, **{name: 24}) == 4, name
    assert _read(lib, kos=500) == 3 and _read(lib, voh=100) == 3
    assert _read(lib, kos=516) == 4
    assert _read(lib, bts=7) == 3
    assert _read(lib, R=-1) == 2 and _read(lib, R=1 << 31) == 2
    assert _read(lib, R=0) == 0 and _read(lib, B=0) == 0


def _attn(lib, options=None, **kw):
    import ctypes

    a = dict(q=256, qs=1024, qh=128, kc=256, vc=256, sk=256, sv=256, nb=10, bs=16, bt=256, bts=8, mb=8, ctx=256,
             qsl=256, B=2, out=512, os=1024, oh=128, T=2, hq=8, hkv=4, d=128, fmt=1, scale=0.1, ws=256, wsb=1 << 20)
    a.update(kw)
    opt = ops.attention_options(options)
    return lib.pkv_paged_attention_q8(a["q"], a["qs"], a["qh"], a["kc"], a["vc"], a["sk"], a["sv"], a["nb"], a["bs"],
                                      a["bt"], a["bts"], a["mb"], a["ctx"], a["qsl"], a["B"], a["out"], a["os"],
                                      a["oh"], a["T"], a["hq"], a["hkv"], a["d"], a["fmt"], a["scale"], a["ws"],
                                      a["wsb"], None, None if opt is None else ctypes.byref(opt))


def test_attention_refusals(lib):
    assert _attn(lib, d=80) == 5 and _attn(lib, bs=48) == 5 and _attn(lib, fmt=7) == 5
    assert _attn(lib, hq=12, hkv=3) == 5 and _attn(lib, hq=36) == 5
    for scale in (0.0, -0.1, float("inf"), float("nan")):
        assert _attn(lib, scale=scale) == 2
    for name in ("q", "kc", "vc", "sk", "sv", "bt", "ctx", "qsl", "out"):
        assert _attn(lib, **{name: None}) == 1, name
    for name in ("q", "kc", "vc", "sk", "sv", "out"):
        assert _attn(lib, **{name: 264}) == 4, name
    assert _attn(lib, os=100) == 3 and _attn(lib, bts=4) == 3
    assert _attn(lib, options={"decode_kernel": "simt"}) == 5
    assert _attn(lib, options={"prefill_kernel": "mma"}) == 5
    assert _attn(lib, T=0) == 0 and _attn(lib, B=0) == 0


def test_binding_refuses_cpu_tensors_and_wrong_types():
    z = torch.zeros(2, 8, 1, 64, dtype=torch.int8)
    s = torch.ones(2, 1)
    with pytest.raises(ValueError, match="CUDA"):
        ops.kv_read_q8(z, z, s, s, None, None, None, None, None)
    with pytest.raises(TypeError, match="int8"):
        ops.kv_read_q8(z.float(), z, s, s, None, None, None, None, None)
    with pytest.raises(TypeError, match="torch.Tensor"):
        ops.kv_read_q8(None, z, s, s, None, None, None, None, None)
    with pytest.raises(TypeError, match="dtype"):
        ops.alloc_q8_cache(2, 16, 1, 64, dtype=torch.bfloat16, device="cpu")
    k, v, ks, vs = ops.alloc_q8_cache(2, 16, 1, 64, dtype=torch.float8_e4m3fn, device="cpu")
    assert k.shape == v.shape == (2, 16, 1, 64) and ks.shape == vs.shape == (2, 1) and ks.dtype == torch.float32
