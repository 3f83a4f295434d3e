"""Helpers for the tests of the 8-bit cache: seeded pools and batches, the comparison with the oracle
and the tolerances, each derived where it is defined."""

import numpy as np
import torch

import oracle
from oracle import q8 as OQ
from paged_kv_gqa_14_gb300 import ops
from paged_kv_gqa_14_gb300 import workloads as W
from tests.gpu_util import bf16_to_dev, dev_to_bits, idx_to_dev, rope_tol

KINDS = ("int8", "e4m3")
DTYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
EVERY_CODE_BUT_NAN = {"int8": np.arange(256, dtype=np.uint8),
                      "e4m3": np.array([c for c in range(256) if c & 127 != 127], dtype=np.uint8)}


def pool(rng, num_blocks, bs, hkv, d, kind, spread=6, poison=True, used=None):
    """Bytes and scales of a pool: any finite code, scales 2^(-7 - spread .. -7 + spread).  With `poison`, rows
    not marked in `used` [num_blocks, bs] are NaN (e4m3) or the extreme -128 (int8)."""
    codes = rng.choice(EVERY_CODE_BUT_NAN[kind], size=(num_blocks, bs, hkv, d))
    if kind == "int8":
        codes = np.where(codes == 128, np.uint8(129), codes)  # -128 is never written
    else:
        codes = np.where(rng.random(codes.shape) < 0.5, codes & 0x3F | codes & 0x80, codes)  # mostly below 2
    if poison and used is not None:
        codes[~used] = 0x7F if kind == "e4m3" else 0x80
    scale = np.ldexp(1.0, rng.integers(-7 - spread, -6 + spread, size=(num_blocks, hkv)))
    return codes.astype(np.uint8), scale.astype(np.float32)


class Q8:
    """A batch over an 8-bit cache, on the host and on the GPU.  `fresh`: before its append (the rows of
    the step's tokens hold poison, the scales of blocks without earlier rows NaN); else after it."""

    def __init__(self, ctx, spans, hq, hkv, d, bs, kind, seed, spread=2, num_blocks=None, extra_tokens=0,
                 fresh=False):
        rng = np.random.default_rng(seed)
        ctx, spans = np.asarray(ctx, np.int64), np.asarray(spans, np.int64)
        self.kind, self.bs = kind, bs
        pages = -(-ctx // bs)
        nb = int(pages.sum()) + 3 if num_blocks is None else num_blocks
        perm = rng.permutation(nb)
        self.bt = np.full((len(ctx), max(1, int(pages.max(initial=0)) + 1)), -1, np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.bt[b, :n] = perm[at:at + n]
            at += n
        self.ctx, self.qsl = ctx.astype(np.int32), np.concatenate([[0], np.cumsum(spans)]).astype(np.int32)
        self.T = int(spans.sum()) + extra_tokens
        self.d, self.hq, self.hkv, self.theta, self.scale = d, hq, hkv, 1.0e6, float(d**-0.5)
        self.q, self.k, self.v = (W.normal_bf16(rng, (self.T, h, d)) for h in (hq, hkv, hkv))
        # rows that hold context before the step
        self.old = np.zeros((nb, bs), bool)
        self.seen = np.zeros((nb, bs), bool)
        for b in range(len(ctx)):
            for p in range(int(ctx[b])):
                self.seen[self.bt[b, p // bs], p % bs] = True
                self.old[self.bt[b, p // bs], p % bs] = p < ctx[b] - spans[b]
        used = self.old if fresh else self.seen
        self.kc, self.ks = pool(rng, nb, bs, hkv, d, kind, spread, used=used)
        self.vc, self.vs = pool(rng, nb, bs, hkv, d, kind, spread, used=used)
        self.ks[~used.any(1)] = self.vs[~used.any(1)] = np.nan

    def to_dev(self):
        self.g_q, self.g_k, self.g_v = (bf16_to_dev(x) for x in (self.q, self.k, self.v))
        self.g_bt, self.g_ctx, self.g_qsl = (idx_to_dev(x) for x in (self.bt, self.ctx, self.qsl))
        self.g_kc, self.g_vc = (idx_to_dev(x.view(np.int8)).view(DTYPE[self.kind]) for x in (self.kc, self.vc))
        self.g_ks, self.g_vs = (idx_to_dev(x) for x in (self.ks, self.vs))
        return self

    @property
    def cache(self):
        return self.g_kc, self.g_vc, self.g_ks, self.g_vs

    def append(self, **kw):
        ops.kv_append_q8(self.g_q, self.g_k, self.g_v, self.g_bt, self.g_ctx, self.g_qsl, *self.cache, self.theta, **kw)

    def attend(self, out=None, **kw):
        return ops.paged_attention_q8(self.g_q, *self.cache, self.g_bt, self.g_ctx, self.g_qsl, self.scale, out=out, **kw)

    def oracle_append(self):
        return OQ.kv_append_q8(self.q, self.k, self.v, self.bt, self.ctx, self.qsl, self.kc, self.vc, self.ks, self.vs,
                               self.theta, self.kind)

    def oracle_attention(self, q=None, kc=None, vc=None, ks=None, vs=None):
        """(rows, allowed error) of the attention over what the cache stands for."""
        q = self.q if q is None else q
        k = OQ.dequantise(self.kc if kc is None else kc, self.ks if ks is None else ks, self.kind)
        v = OQ.dequantise(self.vc if vc is None else vc, self.vs if vs is None else vs, self.kind)
        args = (self.bt, self.ctx, self.qsl, self.scale)
        ref = oracle.paged_attention(q, k, v, *args)
        size, total = value_sizes(q, k, v, *args)
        return ref, attention_tol(ref, size, total, score_bound(q, k, self.bt, self.ctx, self.scale))


def value_sizes(q, k, v, bt, ctx, qsl, scale):
    """For every output, over the keys its row sees: sum(weight |v|) and sum(|v|) (the mean that a zero
    query gives, times the number of keys)."""
    size = oracle.paged_attention(q, k, v & np.uint16(0x7FFF), bt, ctx, qsl, scale)
    mean = oracle.paged_attention(np.zeros_like(q), k, v & np.uint16(0x7FFF), bt, ctx, qsl, scale)
    seen = np.zeros(q.shape[0])
    for b in range(len(ctx)):
        n = int(qsl[b + 1] - qsl[b])
        seen[int(qsl[b]):int(qsl[b + 1])] = int(ctx[b]) - n + 1 + np.arange(n)
    return size, mean * seen[:, None, None]


def score_bound(q, k_bits, bt, ctx, scale):
    """The largest sum over d of |q k| scale that any row and any key of the batch can have."""
    qn = np.sqrt((oracle.bf16_bits_to_f64(q) ** 2).sum(-1)).max(initial=0.0)
    bs = k_bits.shape[1]
    kn = 0.0
    for b, n in enumerate(ctx):
        x = oracle.bf16_bits_to_f64(k_bits[bt[b, : -(-int(n) // bs)]]).reshape(-1, *k_bits.shape[2:])[: int(n)]
        kn = max(kn, np.sqrt((x**2).sum(-1)).max(initial=0.0))
    return qn * kn * scale


def attention_tol(ref, size, total, smax):
    """Allowed |gpu - oracle| of an attention output, from the kernel's roundings:

    * the bf16 output: half a step, 2^-8 |ref|;
    * a weight p rounded to f16: half a step, 2^-11 p, so at most 2^-11 sum(w |v|) = 2^-11 size; where p is
      below f16's normal range half a step is 2^-25, the row's largest weight being 2^7 or more (m is the
      maximum of some of its keys, and p = 2^(s - m + 7)), so that after the division it is at most 2^-32,
      and over the keys at most 2^-32 sum(|v|) = 2^-32 total;
    * a score s' = s log2(e), |s| <= smax: 128 products summed in fp32 (each step of a tensor-core sum
      may truncate: 2^-23 of the running magnitude, 128 + 3 of them), q's f16 form (2^-39 of its
      largest component a product), the factor's and the subtraction's rounding (2^-22 s'), ex2.approx
      (2^-22): a weight is off by ln 2 * s' * 2^-15.9 + 2^-21 relatively, hence 2^-15.5 smax + 2^-21, in the
      numerator and in the sum alike (twice);
    * the fp32 sums over keys: each weight's error 2^-23 a step at most, over at most 2^12 keys here
      added in units of 16, 2^-14.
    """
    eps = 2.0**-11 + 2 * (2.0**-15.5 * max(smax, 1.0) + 2.0**-21) + 2 * 2.0**-14
    return 2.0**-8 * np.abs(ref) + eps * size + 2.0**-32 * total + 1e-37


def assert_attention(got, ref, tol, covered=None):
    got = got.float().cpu().numpy().astype(np.float64)
    if covered is not None:
        got, ref, tol = got[covered], ref[covered], tol[covered]
    assert np.all(np.isfinite(got)), "non-finite output"
    over = np.abs(got - ref) / tol
    assert over.max(initial=0.0) <= 1.0, f"{over.max():.2f} times the allowed error at {np.unravel_index(over.argmax(), over.shape)}"


def near_border(exact, kind, eps):
    """Where a value x / scale lies within eps (an array) of a border between two held values."""
    a = np.abs(exact)
    if kind == "int8":
        return np.abs(a - np.floor(a) - 0.5) <= eps
    _, e = np.frexp(a)
    step = np.ldexp(1.0, np.maximum(e, -5) - 4)
    y = a / step
    return np.abs(y - np.floor(y) - 0.5) * step <= eps


def assert_append(c, ref):
    """The cache after an append against the oracle's: everything equal, but that a K value whose
    exact rotation lies within the kernel's error of a rounding border may go to either neighbour, and q
    within the rotation's bound.  The kernel's K before rounding: 2^-24 |k| + 2^-28 pair (its header)."""
    q_rot, kc, vc, ks, vs, k_exact = ref
    got = {n: t.view(torch.int8).cpu().numpy().view(np.uint8) for n, t in (("k", c.g_kc), ("v", c.g_vc))}
    assert np.array_equal(c.g_vs.cpu().numpy(), vs.astype(np.float32), equal_nan=True), "v_scale"
    assert np.array_equal(c.g_ks.cpu().numpy(), ks.astype(np.float32), equal_nan=True), "k_scale"
    assert np.array_equal(got["v"], vc), "v_cache"
    off = got["k"] != kc
    half = k_exact.shape[-1] // 2
    mag = np.abs(np.nan_to_num(k_exact))
    pair = mag[..., :half] + mag[..., half:]
    # |k_i| + |k_j| of the unrotated pair is at most sqrt(2) times that of the rotated one
    eps = 2.0**-24 * mag + 2.0**-27.4 * np.concatenate([pair, pair], -1)
    assert not (off & ~near_border(np.nan_to_num(k_exact), c.kind, eps)).any(), "k_cache"
    step = np.abs(OQ.decode(got["k"], c.kind) - OQ.decode(kc, c.kind))[off]
    assert (step <= (1 if c.kind == "int8" else 32)).all(), "k_cache: more than one step away"
    covered = np.zeros(c.T, bool)
    covered[: int(c.qsl[-1])] = True
    q_got = dev_to_bits(c.g_q)
    assert np.array_equal(q_got[~covered], c.q[~covered]), "q rows outside every span"
    ref64 = oracle.bf16_bits_to_f64(q_rot)
    err = np.abs(oracle.bf16_bits_to_f64(q_got) - ref64)
    assert (err <= rope_tol(c.q, ref64)).all(), "q"
