"""The 8-bit cache on the GPU at the edges of what its calls take: scales far apart, values that are not
finite, tables that do not add up, late positions.  Tolerances: tests/q8_util.py, or derived at the test."""

import numpy as np
import pytest
import torch

import oracle
from oracle import q8 as OQ
from paged_kv_gqa_14_gb300 import ops
from tests.q8_util import KINDS, Q8, assert_append, assert_attention, attention_tol, score_bound, value_sizes

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word():
    ops.get_device_error()
    yield
    assert ops.get_device_error() == 0, "a device error was left behind"


# ------------------------------------------------------------------------- V scales far apart
def falling(c, exponents, zero_from=None):
    """V scales 2^exponents[i] on the i-th part of every sequence's blocks; zero V from part `zero_from` on."""
    for b, n in enumerate(-(-c.ctx // c.bs)):
        for i, part in enumerate(np.array_split(c.bt[b, :n], len(exponents))):
            c.vs[part] = 2.0 ** exponents[i]
            if zero_from is not None and i >= zero_from:
                c.vc[part] = 0
    return c.to_dev()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hkv,d,bs", [(8, 128, 16), (1, 128, 16), (2, 64, 8), (4, 64, 128)])
@pytest.mark.parametrize("exponents,zero_from", [((20, -40, -100), 2), ((0, -30, -60, -90), None),
                                                 ((20, -40, 20, -40, -100, 20), None)])
def test_decode_over_v_scales_that_fall_step_by_step(kind, hkv, d, bs, exponents, zero_from):
    """Each step is within the 2^80 that sums in units of a scale may come down, all of them together are not: the
    sums stay finite.  One CTA takes every page, so that one warp meets them all."""
    c = falling(Q8([3000, 700], [1, 1], 2 * hkv, hkv, d, bs, kind, seed=hkv, spread=0), exponents, zero_from)
    ref, tol = c.oracle_attention()
    assert_attention(c.attend(options={"decode_ctas": 1}), ref, tol)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,bs", [(128, 16), (64, 128)])
@pytest.mark.parametrize("exponents,zero_from", [((20, -40, -100), 2), ((0, -30, -60, -90), None)])
def test_prefill_over_v_scales_that_fall_from_tile_to_tile(kind, d, bs, exponents, zero_from):
    """The same for a prefill row's one sum, the scales alike in each tile of 128 keys; items enough that no item's
    keys are shared out among CTAs."""
    n = 128 * len(exponents)
    c = falling(Q8([n] * 10, [n - 5] * 10, 8, 8, d, bs, kind, seed=d, spread=0), exponents, zero_from)
    ref, tol = c.oracle_attention()
    for options in (None, {"overlap": False}):
        assert_attention(c.attend(options=options), ref, tol)


# ------------------------------------------------------------------- tables that do not add up
@pytest.mark.parametrize("cache", ("int8", "bf16"))
@pytest.mark.parametrize("num_seqs,num_tokens", [(256, 256), (700, 700), (1300, 1300), (20, 300), (1300, 4000)])
@pytest.mark.parametrize("options", (None, {"plan_early": True}))
def test_spans_that_go_back_stay_inside_the_workspace(cache, num_seqs, num_tokens, options):
    """query_start_loc 0, T, 0, T, ..: every second span is the whole batch again.  Only the one before the first
    that goes back is computed, and nothing is written behind the workspace."""
    hq, hkv, d, bs = 2, 1, 64, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(num_tokens, hq, d, generator=g, device="cuda").to(torch.bfloat16)
    width = -(-num_tokens // bs)
    table = torch.arange(width, dtype=torch.int32, device="cuda").repeat(num_seqs, 1)
    ctx = torch.full((num_seqs,), num_tokens, dtype=torch.int32, device="cuda")
    back = torch.tensor([0, num_tokens], dtype=torch.int32, device="cuda").repeat(num_seqs // 2 + 1)[: num_seqs + 1]
    once = torch.full_like(back, num_tokens)
    once[0] = 0
    need = ops.workspace_size(num_tokens, num_seqs, hq, hkv, d, width)
    ws = torch.full((need + (1 << 20),), 0xAB, dtype=torch.uint8, device="cuda")
    if cache == "int8":
        pools = [torch.randint(-100, 100, (width, bs, hkv, d), dtype=torch.int8, generator=g, device="cuda") for _ in "kv"]
        pools += [torch.full((width, hkv), 2.0**-7, device="cuda") for _ in "kv"]
        call = ops.paged_attention_q8
    else:
        pools = [torch.randn(width, bs, hkv, d, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv"]
        call = ops.paged_attention
    outs = []
    for qsl, bits in ((once, 0), (back, 4)):
        outs.append(torch.full_like(q, 3.0))
        call(q, *pools, table, ctx, qsl, 0.1, out=outs[-1], workspace=ws[:need], options=options)
        assert ops.get_device_error() == bits
        assert (ws[need:] == 0xAB).all()
    assert torch.equal(*outs) and not (outs[0] == 3.0).all(-1).any()


@pytest.mark.parametrize("num_tokens,num_seqs,bs", [(1000, 20, 16), (70, 31, 8)])  # numbered by block, by token
def test_starts_that_go_back_put_no_row_before_its_table(num_tokens, num_seqs, bs):
    """A search over starts that go back ends at a sequence that begins behind the token or row: it has no place
    there (its position, and its block table's column, would be negative).  Flagged, and nothing is written
    outside the batch's blocks."""
    c = Q8([40] * num_seqs, [1] * num_seqs, 2, 1, 64, bs, "int8", seed=1, extra_tokens=num_tokens - num_seqs, fresh=True)
    starts = np.full(num_seqs + 1, num_tokens - 10, np.int32)
    starts[[0, -2, -3, -4, -5, -6]] = 0  # six of them are at or below a small token: the search ends at sequence 5
    starts[6] = num_tokens - 6
    c.qsl = starts
    c.ctx[5] = 5
    c.to_dev()
    before = [t.clone() for t in (*c.cache, c.g_q)]
    c.append()
    assert ops.get_device_error() == 4
    unused = torch.from_numpy(np.setdiff1d(np.arange(c.kc.shape[0]), c.bt)).cuda()
    for a, b in zip(before, c.cache):
        assert torch.equal(a[unused].view(torch.uint8), b[unused].view(torch.uint8))
    out = [torch.zeros(num_tokens, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    ops.kv_read_q8(*c.cache, c.g_bt, c.g_ctx, c.g_qsl, *out)
    assert ops.get_device_error() == 4
    assert not out[0][: num_tokens - 10].any() and not out[1][: num_tokens - 10].any()
    kb, vb = (torch.zeros(c.kc.shape, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    pos, slots = (torch.zeros(num_tokens, dtype=torch.int64, device="cuda") for _ in "ps")
    ops.kv_append_paged(c.g_q, c.g_k, c.g_v, c.g_bt, c.g_ctx, c.g_qsl, kb, vb, c.theta, positions_out=pos,
                        slot_mapping_out=slots)
    assert ops.get_device_error() == 4
    assert (slots[: num_tokens - 10] == -1).all() and not kb[unused].any()


# ------------------------------------------------------------------------ steps that start early
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hkv,d,bs", [(1, 64, 8), (1, 128, 16), (2, 64, 16), (2, 128, 128), (4, 64, 8), (8, 128, 16)])
@pytest.mark.parametrize("batch", ("few units", "units past the stages", "more sequences than a scan", "longer spans"))
def test_steps_that_start_early_give_the_same_bits(kind, hkv, d, bs, batch):
    """Decode steps (no planner kernel) right after their append, whose growing values rescale every newest block,
    between blocks of other sequences: each step's rows and the cache in the end are those of the calls that wait
    for the append, eager and in a graph."""
    rng = np.random.default_rng(hkv + bs)
    n, hi = {"few units": (40, 200), "units past the stages": (24, 3000), "more sequences than a scan": (900, 60),
             "longer spans": (30, 400)}[batch]
    ctx = rng.integers(12, hi, size=n)
    spans = np.ones(n, np.int64)
    if batch == "longer spans":  # no more tokens than sequences
        spans[[3, 9, 20]] = 0, 3, 0
        spans[25] = 0
    options = {"decode_ctas": 7} if batch == "units past the stages" else {}
    steps = 5
    c = Q8(ctx, spans, 2 * hkv, hkv, d, bs, kind, seed=bs, fresh=True).to_dev()
    c.g_ctx -= steps - 1
    start = [t.clone() for t in (*c.cache, c.g_ctx)]
    qs = [torch.randn_like(c.g_q.float()).to(torch.bfloat16) for _ in range(steps)]
    kvs = [[(torch.randn_like(c.g_k.float()) * 2.0**i).to(torch.bfloat16) for _ in "kv"] for i in range(steps)]
    ws = ops.alloc_workspace(c.T, n, 2 * hkv, hkv, d, c.bt.shape[1], decode_ctas=options.get("decode_ctas", 0))

    def run(outs, opt):
        for t, s in zip((*c.cache, c.g_ctx), start):
            t.copy_(s)
        for i in range(steps):
            c.g_q.copy_(qs[i])
            c.g_k, c.g_v = kvs[i]
            c.append()
            c.attend(out=outs[i], workspace=ws, options=opt)
            c.g_ctx += 1

    want = [torch.zeros_like(c.g_q) for _ in range(steps)]
    run(want, ops.attention_options(options))
    held = [t.clone() for t in c.cache]
    for flag in ("plan_early", "stream_early"):
        opt = ops.attention_options({flag: True, **options})
        got = [torch.zeros_like(c.g_q) for _ in range(steps)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(got, opt)
        for eager in (True, False):
            for g in got:
                g.zero_()
            run(got, opt) if eager else graph.replay()
            for i, (a, b) in enumerate(zip(want, got)):
                assert torch.equal(a.view(torch.int16), b.view(torch.int16)), f"{flag}, step {i}"
            for a, b in zip(held, c.cache):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ------------------------------------------------------------------- values that are not numbers
@pytest.mark.parametrize("d,bs", [(64, 8), (128, 16), (128, 128)])
@pytest.mark.parametrize("group", (1, 3, 8))
@pytest.mark.parametrize("many", (False, True))  # items whose keys CTAs share, and items enough for every CTA
def test_a_nan_among_the_values_reaches_only_rows_that_see_it(d, bs, group, many):
    """NaN held in V (the append holds one so in e4m3): every row whose position is at or behind it is NaN in its
    column, every other output is what it would be without."""
    hkv = 8 if many else 2
    ctx, spans = [300, 129, 40, 140, 513, 77], [200, 129, 1, 3, 33, 77]
    if many:
        ctx, spans = ctx * 4, spans * 4
    c = Q8(ctx, spans, group * hkv, hkv, d, bs, "e4m3", seed=d + group)
    rng = np.random.default_rng(group)
    for b, (n, m) in enumerate(zip(ctx, spans)):
        # the first and the last new token, one between them, one before the span and others anywhere
        for p in {n - m, n - 1, n - m + m // 2, max(0, n - m - 5), *rng.integers(0, n, size=2)}:
            if b % 6 != 5 or p == n - 1:  # (the last sequence has one in its last token alone)
                c.vc[c.bt[b, p // bs], p % bs, rng.integers(hkv), rng.integers(d)] = rng.choice([0x7F, 0xFF])
    c.to_dev()
    ref, tol = c.oracle_attention()
    bad = np.isnan(ref)
    assert bad.any() and not bad.all(-1).any()
    for options in (None, {"overlap": False}):
        got = c.attend(options=options).float().cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isnan(got), bad)
        assert (np.abs(got - ref)[~bad] <= tol[~bad]).all()


# ------------------------------------------------------------------------------- another stream
@pytest.mark.parametrize("cache", ("int8", "bf16"))
def test_a_workspace_made_for_another_stream_stays_with_it(cache, monkeypatch):
    """The workspace of a call on another stream is freed when the call returns, before its kernels have run: the
    current stream's next tensors must not get its memory."""
    c = Q8([900, 70], [1, 40], 4, 2, 64, 16, "int8", seed=1).to_dev()
    made = []
    alloc = ops.alloc_workspace
    monkeypatch.setattr(ops, "alloc_workspace", lambda *a, **kw: made.append(alloc(*a, **kw)) or made[-1])
    if cache == "int8":
        def call(**kw):
            return c.attend(**kw)
    else:
        pools = [torch.randn(*c.kc.shape, device="cuda").to(torch.bfloat16) for _ in "kv"]

        def call(**kw):
            return ops.paged_attention(c.g_q, *pools, c.g_bt, c.g_ctx, c.g_qsl, c.scale, **kw)

    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    made.clear()
    out = call(stream=side)
    at, size = made[0].data_ptr(), made[0].numel()
    made.clear()
    later = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert at not in [t.data_ptr() for t in later]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)


# ------------------------------------------------------------------------ the longest contexts
@pytest.mark.parametrize("cache", ("int8", "bf16"))
@pytest.mark.parametrize("num_tokens", (1, 2))  # a decode step, a prefill span
def test_contexts_whose_tiles_would_pass_2_31_are_flagged(cache, num_tokens):
    """Keys are counted in 32 bits, rounded up to whole tiles: contexts above 2^31 - 4096 are skipped."""
    bs, width = 128, 1 << 24
    table = torch.zeros(1, width, dtype=torch.int32, device="cuda")
    q = torch.zeros(num_tokens, 2, 64, dtype=torch.bfloat16, device="cuda")
    qsl = torch.tensor([0, num_tokens], dtype=torch.int32, device="cuda")
    if cache == "int8":
        pools = [torch.zeros(1, bs, 1, 64, dtype=torch.int8, device="cuda") for _ in "kv"]
        pools += [torch.ones(1, 1, device="cuda") for _ in "kv"]
        call = ops.paged_attention_q8
    else:
        pools = [torch.zeros(1, bs, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        call = ops.paged_attention
    for ctx in (2**31 - 1, 2**31 - 4095):
        out = torch.full_like(q, 3.0)
        call(q, *pools, table, torch.tensor([ctx], dtype=torch.int32, device="cuda"), qsl, 0.1, out=out)
        assert ops.get_device_error() == 8
        assert (out == 3.0).all()


# ------------------------------------------------------------------------ batches mostly empty
def test_read_passes_over_a_million_sequences_without_rows():
    """Rows of one warp that belong to the first, a middle and the last of 2^20 sequences, the others without any:
    found without walking over them (which took 42 ms)."""
    n = 1 << 20
    c = Q8([40], [1], 2, 2, 64, 16, "int8", seed=1).to_dev()
    lens = np.zeros(n, np.int64)
    lens[[0, n // 3, n - 1]] = 3, 2, 4
    rsl = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()
    table, ctx = c.g_bt.expand(n, -1).contiguous(), c.g_ctx.expand(n).contiguous()
    out = [torch.zeros(9, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    want = [torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    one = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    ops.kv_read_q8(*c.cache, c.g_bt, c.g_ctx, one, *want)
    times = []
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in "ab")
        a.record()
        ops.kv_read_q8(*c.cache, table, ctx, rsl, *out)
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b))
    for o, w in zip(out, want):
        assert torch.equal(o[:3], w[1:]) and torch.equal(o[3:5], w[2:]) and torch.equal(o[5:], w)
    assert min(times) < 2.0, f"{min(times)} ms"


# ------------------------------------------------------------------------ rotation and rounding
# An append rounds a rotated k as a value within 2^-27 (|k_i| + |k_{i+d/2}|) of the exact rotation is (include/pkv.h):
#   the angle's rest |d| <= pi/256 in fp32: its conversion, constant and product 2.6 2^-31 (half a step of 2^-31 at
#   this size each, the constant 2^-25.1 off); the frequency's last unit, 2^-64 of a turn times a position below 2^31,
#   1.6 2^-31; its sine, the two products with it and the sum with the table's low part 4 2^-31: each of sine and cosine
#   within 8.2 2^-31;
#   the two low products (|y| 0.0123 of it, half a step 2^-24 relative) and their sum with the high products' rest
#   3 * 1.6 2^-31 (|x| + |y|);
# together 13 2^-31 < 2^-27.  Nothing else is rounded before the eight bits.
ROTATION = 2.0**-27


def rotated(x, pos, theta):
    """x [T, H, d] fp64 turned by the angles of positions `pos` (fp64; the turn modulo one is exact in integers),
    and |x_i| + |x_{i+d/2}|."""
    d = x.shape[-1]
    turn = pos[:, None] * torch.from_numpy(ops.rope_turn_table(theta, d).view(np.int64)).cuda()  # modulo 2^64
    a = (turn.double() * (2 * np.pi / 2.0**64))[:, None, :]
    lo, hi = x[..., : d // 2], x[..., d // 2:]
    pair = lo.abs() + hi.abs()
    return (torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1), torch.cat([pair, pair], -1))


def two_to(e):
    """2^e in fp64, exactly (torch.ldexp goes through a rounded power)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def steps(y, kind):
    """The distance between held values around y."""
    if kind == "int8":
        return torch.ones_like(y)
    return two_to(torch.frexp(y)[1].clamp(min=-5) - 4)


def assert_held(got, exact, scale, pair, kind):
    """Held values `got` against exact / scale rounded to nearest even: either neighbour where the rotation's bound
    reaches a border.  Returns where it does not, and how many went the other way."""
    y = exact / scale
    s = steps(y, kind)
    want = (torch.round(y / s) * s).clamp(-448 if kind == "e4m3" else -127, 448 if kind == "e4m3" else 127)
    at = (y / s).abs()
    sure = ((at - at.floor() - 0.5).abs() * s) > ROTATION * pair / scale
    off = got != want
    assert not (off & sure).any(), f"{int((off & sure).sum())} values on the wrong side of a border"
    assert ((got - want).abs() <= s).all()
    return sure, int(off.sum())


@pytest.mark.parametrize("kind", KINDS)
def test_a_key_is_rounded_as_its_exact_rotation_is(kind):
    """16.8 million keys: no rounding to fp32 comes between (which alone would put some on the other side)."""
    B, n, hkv, d, bs = 64, 2048, 2, 64, 16
    g = torch.Generator(device="cuda").manual_seed(5)
    k = torch.randn(B * n, hkv, d, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.zeros(B * n, hkv, d, dtype=torch.bfloat16, device="cuda")
    cache = ops.alloc_q8_cache(B * n // bs, bs, hkv, d, torch.int8 if kind == "int8" else torch.float8_e4m3fn)
    table = torch.arange(B * n // bs, dtype=torch.int32, device="cuda").view(B, -1)
    ctx = torch.full((B,), n, dtype=torch.int32, device="cuda")
    qsl = torch.arange(B + 1, dtype=torch.int32, device="cuda") * n
    ops.kv_append_q8(q, k, k, table, ctx, qsl, *cache, 1e6)
    exact, pair = rotated(k.double(), torch.arange(n, device="cuda").repeat(B), 1e6)
    exact, pair = (x.view(-1, bs, hkv, d) for x in (exact, pair))
    top = exact.abs().amax((1, 3)) / (127 if kind == "int8" else 448)
    m, e = torch.frexp(top)
    scale = two_to(torch.where(m == 0.5, e - 1, e))
    assert torch.equal(cache[2].double(), scale)
    scale = scale[:, None, :, None]
    sure, other = assert_held(cache[0].float().double(), exact, scale, pair, kind)
    assert other <= 8
    first = exact.float().double() / scale  # rounded to fp32 before
    s = steps(exact / scale, kind)
    assert ((torch.round(first / s) != torch.round(exact / scale / s)) & sure).any(), "the inputs would show it"


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,theta", [(128, 1e6), (64, 10000.0), (64, 0.1)])
def test_append_at_positions_up_to_2_31(kind, d, theta):
    bs, hq, hkv, n = 128, 4, 2, 6
    ends = [2**31 - 1, 2**30 + 77, 2**24 + 5]
    table = torch.full((len(ends), 1 << 24), -1, dtype=torch.int32, device="cuda")
    for b, end in enumerate(ends):
        table[b, (end - n) // bs], table[b, (end - 1) // bs] = 2 * b, 2 * b + ((end - n) // bs != (end - 1) // bs)
    g = torch.Generator(device="cuda").manual_seed(d)
    q, k, v = (torch.randn(3 * n, h, d, generator=g, device="cuda").to(torch.bfloat16) for h in (hq, hkv, hkv))
    cache = ops.alloc_q8_cache(6, bs, hkv, d, torch.int8 if kind == "int8" else torch.float8_e4m3fn)
    for t in cache:
        t.view(torch.uint8).zero_()
    cache[2].fill_(2.0**-100), cache[3].fill_(2.0**-100)
    ctx = torch.tensor(ends, dtype=torch.int32, device="cuda")
    qsl = torch.arange(4, dtype=torch.int32, device="cuda") * n
    q0 = q.double()
    ops.kv_append_q8(q, k, v, table, ctx, qsl, *cache, theta)
    pos = torch.cat([torch.arange(end - n, end, device="cuda") for end in ends])
    block = table[torch.arange(3, device="cuda").repeat_interleave(n), pos // bs].long()
    exact, pair = rotated(k.double(), pos, theta)
    scale = cache[2][block].double()[:, :, None]
    assert_held(cache[0].float().double()[block, pos % bs], exact, scale, pair, kind)
    # the scale holds every value of the block, half of it does not
    top = torch.stack([exact[block == b].abs().amax((0, 2)) for b in block.tolist()])
    top, s = top / (127 if kind == "int8" else 448), scale[:, :, 0]
    assert ((top <= s) & (top > s / 2)).all()
    scale = cache[3][block].double()[:, :, None]
    assert_held(cache[1].float().double()[block, pos % bs], v.double(), scale, torch.zeros_like(exact), kind)
    # q: fp32 (its table entry and three roundings, 2^-22 of the pair), then half a bf16 step, of either side 2^-8
    exact, pair = rotated(q0, pos, theta)
    assert ((q.double() - exact).abs() <= 2.0**-8 * exact.abs() + 2.0**-22 * pair).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bs", (16, 32, 128))
def test_values_that_are_not_finite_beside_rows_that_are_rescaled(kind, bs):
    """Infinities and NaN in blocks of more new rows than are held at a time, and in blocks whose rows before them are
    rounded to a scale that grows: they take no part in it."""
    c = Q8([3 * bs // 4 + 3 * bs, 2 * bs, bs // 2 + 1], [3 * bs, bs + bs // 2, 1], 2, 1, 64, bs, kind, seed=bs, fresh=True)
    grow = np.ldexp(1.0, np.arange(c.T) % 7)[:, None, None]
    c.k, c.v = (oracle.f64_to_bf16_bits(oracle.bf16_bits_to_f64(x) * grow) for x in (c.k, c.v))
    rng = np.random.default_rng(bs)
    bad = {"k": [], "v": []}
    for t in [0, 1, bs // 4, bs, 2 * bs - 1, c.T - 2, c.T - 1]:
        for name, x in (("k", c.k), ("v", c.v)):
            for col, bits in zip(rng.choice(32, 3, replace=False), (0x7F80, 0xFF80, 0x7FC0)):
                x[t, 0, col] = bits
                bad[name].append((t, col, bits))
    c.to_dev().append()
    assert ops.get_device_error() == 0x20
    for t, col, _ in bad["k"]:
        c.k[t, 0, [col, col + 32]] = 0
    for t, col, _ in bad["v"]:
        c.v[t, 0, col] = 0
    ref = list(c.oracle_append())
    b = np.searchsorted(c.qsl, np.arange(c.T), side="right") - 1
    pos = c.ctx[b] - c.qsl[b + 1] + np.arange(c.T)
    for name, i, got in (("k", 1, c.g_kc), ("v", 2, c.g_vc)):
        got = got.view(torch.int8).cpu().numpy().view(np.uint8)
        for t, col, bits in bad[name]:
            place = c.bt[b[t], pos[t] // bs], pos[t] % bs, 0
            for at in (col, col + 32) if name == "k" else (col,):
                code = got[(*place, at)]
                if name == "v" and bits != 0x7FC0:
                    assert code == {("int8", 0x7F80): 127, ("int8", 0xFF80): 129, ("e4m3", 0x7F80): 0x7E,
                                    ("e4m3", 0xFF80): 0xFE}[kind, bits]
                elif kind == "int8":
                    assert code == 0
                else:
                    assert code & 0x7F == 0x7F
                ref[i][(*place, at)] = code
    assert_append(c, ref)


# ------------------------------------------------------------------------------- large scores
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("power", (17, 20, 22, 23, 24, 25, 27, 30))
@pytest.mark.parametrize("sign", (1, -1))
def test_scores_past_what_fp32_holds_to_a_unit(kind, power, sign):
    """Scores of 2^20 to 2^33 (all of them positive, or negative): the largest by far takes all of the softmax.  It is
    key 0's until, from key 150 on, a larger one.  Decode rows and prefill rows, the latter's items shared or not."""
    for spans in ([1, 1, 200], [250] * 12 + [1]):
        ctx = [300, 120, 280] if len(spans) == 3 else [290] * 13
        c = Q8(ctx, spans, 16, 8, 64, 16, kind, seed=power, spread=0)
        q = np.sign(oracle.bf16_bits_to_f64(c.q[:1])) * (1 + np.arange(64) / 64)
        q[q == 0] = 1
        q[:, 1::2] = q[:, ::2]  # the two heads of a group alike
        c.q = oracle.f64_to_bf16_bits(np.repeat(q, c.T, 0) * 2.0**power)
        way = np.sign(q[0, ::2])  # [hkv, 64]
        rng = np.random.default_rng(power)
        for b, n in enumerate(ctx):
            for p in range(n):
                size = {0: 30.0, 150: 112.0}.get(p, float(rng.integers(1, 12)))
                if sign < 0:
                    size = {30.0: -28.0, 112.0: -2.0}.get(size, -100.0 + size)
                c.kc[c.bt[b, p // 16], p % 16] = OQ.encode(way * size, kind)
        c.ks[:] = np.where(np.isnan(c.ks), c.ks, 2.0**-7)
        c.to_dev()
        v = oracle.bf16_bits_to_f64(OQ.dequantise(c.vc, c.vs, kind))
        for options in (None, {"overlap": False}):
            got = c.attend(options=options).float().cpu().numpy().astype(np.float64)
            for b, n in enumerate(ctx):
                m = spans[b]
                for r in range(m):
                    key = 150 if n - m + r >= 150 else 0
                    want = np.repeat(v[c.bt[b, key // 16], key % 16], 2, axis=0)
                    # a weight's f16 rounding, 2^-11, and the output's, 2^-8
                    err = np.abs(got[c.qsl[b] + r] - want)
                    assert (err <= (2.0**-8 + 2.0**-11) * np.abs(want)).all(), (b, r)


# --------------------------------------------------------------- scales far apart inside a tile
@pytest.mark.parametrize("kind,apart", [("int8", 29), ("e4m3", 20)])
@pytest.mark.parametrize("d,bs", [(64, 8), (128, 16), (64, 64)])
@pytest.mark.parametrize("small_first", (True, False))
def test_prefill_is_exact_to_the_edge_of_what_a_tile_holds(kind, apart, d, bs, small_first):
    """Among 128 keys the scales of K and of V lie 2^29 (int8) or 2^20 (e4m3) apart: each row is as near as ever, rows
    that see only the small blocks included (their scores are of the size of one)."""
    c = Q8([128, 300], [128, 260], 4, 2, d, bs, kind, seed=d + bs, spread=0)
    for b, n in enumerate(-(-c.ctx // bs)):
        small = (np.arange(n) < max(1, n // 3)) == small_first
        for s in (c.ks, c.vs):
            s[c.bt[b, :n][~small]] = 2.0 ** (-7 + apart)
            s[c.bt[b, :n][small]] = 2.0**-7
    c.to_dev()
    k, v = OQ.dequantise(c.kc, c.ks, kind), OQ.dequantise(c.vc, c.vs, kind)
    args = (c.bt, c.ctx, c.qsl, c.scale)
    ref = oracle.paged_attention(c.q, k, v, *args)
    size, total = value_sizes(c.q, k, v, *args)
    got = c.attend().float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    for b in range(2):
        first = int(c.ctx[b] - (c.qsl[b + 1] - c.qsl[b]))
        n = -(-int(c.ctx[b]) // bs)
        edge = max(1, n // 3) * bs  # the first keys of the other scale
        r = np.arange(c.qsl[b], c.qsl[b + 1])
        seen = r - c.qsl[b] + first
        for rows, keys in ((r[seen < edge], edge), (r[seen >= edge], int(c.ctx[b]))):
            if len(rows) == 0:
                continue
            smax = score_bound(c.q[rows], k, c.bt[b:b + 1], np.array([min(keys, int(c.ctx[b]))]), c.scale)
            tol = attention_tol(ref[rows], size[rows], total[rows], smax)
            over = np.abs(got[rows] - ref[rows]) / tol
            assert over.max() <= 1, (b, keys, over.max())


# ------------------------------------------------------------------------------- bounded waits
@pytest.mark.parametrize("shared", (True, False))
def test_prefill_waits_run_out_and_report(shared):
    """The producer issues nothing: every other role's wait runs out (about a second, once for a CTA), CTAs that share
    an item meet at the cluster's barriers all the same, the error is reported and the next call runs as ever."""
    c = Q8([200, 300], [60, 1], 4, 2, 64, 16, "e4m3", seed=1) if shared else Q8([290] * 13, [250] * 12 + [1], 16, 8, 64, 16,
                                                                               "int8", seed=1)
    c.to_dev()
    want = c.attend()
    ops.set_fault_injection("prefill_no_copies")
    try:
        got = c.attend()
        assert ops.get_device_error() == 0x10
    finally:
        ops.set_fault_injection(None)
    assert torch.equal(got[-1], want[-1])  # the decode row
    assert torch.equal(c.attend(), want)
