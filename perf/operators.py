"""The operators of the 8-bit KV cache as they are measured: cases, inputs, a plain form in torch
and the calls of this package.

The cache: k_cache and v_cache [num_blocks, block_size, Hkv, d] in int8 or float8_e4m3fn, and one
power-of-two scale for each block and kv head, k_scale and v_scale float32 [num_blocks, Hkv]; a
held value x stands for x * scale.  A block's scale is the smallest power of two (2^-100 at least)
with which its largest magnitude fits the type (127, 448); when later tokens of the block need a
larger one, the rows already there are rounded to it.

  append     RoPE of the new tokens' q and k, and k and v quantised into the paged cache; then the
             blocks the step touched are read back as bf16 (what the cache stands for)
  read       the last tokens of every sequence, read back from the cache as bf16
  attention  grouped-query attention of the new tokens over the 8-bit cache, decode tokens and
             causal prefill chunks in one call
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
LARGEST = {"int8": 127.0, "e4m3": 448.0}
THETA = 1.0e6


def _case(op, dtype, hq, hkv, d, bs, dec=0, lo=1, hi=1, pre=0, chunk=0, prior=0, lens=0):
    """dec sequences of one new token with contexts in [lo, hi]; pre sequences with chunks of up to
    `chunk` new tokens behind up to `prior` cached ones; `lens` seeds the lengths."""
    return {"op": op, "dtype": dtype, "hq": hq, "hkv": hkv, "d": d, "bs": bs, "dec": dec, "lo": lo, "hi": hi,
            "pre": pre, "chunk": chunk, "prior": prior, "lens": lens}


def listed():
    cases = {
        # one decode step's append of a small engine: a handful of launches, latency alone
        "append-32": _case("append", "e4m3", 14, 2, 64, 16, dec=32, lo=129, hi=1152, lens=1),
        # one decode step's append at 256 concurrent sequences: a block rescaled here and there
        "append-256": _case("append", "int8", 16, 8, 128, 16, dec=256, lo=100, hi=2048, lens=2),
        # a full 8192-token budget of prompts: whole blocks are quantised at once
        "append-prompts": _case("append", "int8", 16, 8, 128, 16, pre=5, chunk=2048, prior=700, lens=3),
        # a few short sequences moved out of the 8-bit cache
        "read-short": _case("read", "int8", 14, 2, 64, 16, dec=32, lo=129, hi=1152, lens=4),
        # 50 long contexts read back whole (a cache moved to a 16-bit pool): bandwidth alone
        "read-50x8k": _case("read", "e4m3", 28, 4, 128, 32, dec=50, lo=8000, hi=8192, lens=5),
        # the smallest attention call: four short contexts
        "attn-4": _case("attention", "int8", 4, 2, 64, 16, dec=4, lo=1, hi=100, lens=6),
        # a small decode batch, head_dim 64, a group of seven
        "attn-32": _case("attention", "e4m3", 14, 2, 64, 16, dec=32, lo=129, hi=1152, lens=7),
        # 256 decode sequences of up to 2048 tokens: the serving step that the cache's width decides
        "attn-256": _case("attention", "int8", 16, 8, 128, 16, dec=256, lo=100, hi=2048, lens=8),
        # long contexts, a group of seven
        "attn-50x8k": _case("attention", "e4m3", 28, 4, 128, 16, dec=50, lo=8192, hi=8192, lens=9),
        # one user with a very long context: the split over the keys alone fills the GPU
        "attn-1x128k": _case("attention", "int8", 32, 8, 128, 64, dec=1, lo=131000, hi=131072, lens=10),
        # a mixed step: 200 decode tokens beside four prefill chunks
        "attn-mixed": _case("attention", "int8", 16, 8, 128, 16, dec=200, lo=64, hi=2048, pre=4, chunk=512,
                            prior=1536, lens=11),
        # a long prompt's late chunk: compute alone
        "attn-chunk-16k": _case("attention", "e4m3", 28, 4, 128, 32, pre=1, chunk=4096, prior=12288, lens=12),
    }
    return [dict(c, name=n) for n, c in cases.items()]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["append", "read", "attention", "attention"])
        hkv = rng.choice([1, 2, 4, 8])
        group = rng.randint(1, 8)
        c = _case(op, rng.choice(["int8", "e4m3"]), hkv * group, hkv, rng.choice([64, 128]),
                  rng.choice([8, 16, 32, 64, 128]), lens=rng.randint(100, 10**6))
        kind = rng.choice(["dec", "dec", "pre", "mixed"]) if op != "read" else "dec"
        if kind != "pre":
            c["dec"] = _log(rng, 1, 300)
            c["hi"] = _log(rng, 2, 40000 if c["dec"] < 30 else 8192)
            c["lo"] = max(1, c["hi"] // rng.choice([1, 2, 20]))
        if kind != "dec":
            c["pre"] = rng.randint(1, 5)
            c["chunk"] = _log(rng, 2, 4096)
            c["prior"] = rng.choice([0, _log(rng, 1, 12000)])
        w = work(c)
        if w["bytes"] < 1.0e9 and w["flops"] < 7e11 and _padded(c) < 1.6e9:
            return c


def _lens(case):
    """Context lengths (with the step's new tokens) and new tokens of each sequence, decode
    sequences first; part of the case, whatever the seed of the values."""
    rng = np.random.default_rng(case["lens"])
    ctx = rng.integers(case["lo"], case["hi"], size=case["dec"], endpoint=True)
    new = np.ones(case["dec"], np.int64)
    if case["pre"]:
        chunk = rng.integers(max(2, case["chunk"] * 3 // 4), case["chunk"], size=case["pre"], endpoint=True)
        prior = rng.integers(case["prior"] // 2, case["prior"], size=case["pre"], endpoint=True)
        prior[0] = case["prior"]
        ctx = np.concatenate([ctx, prior + chunk])
        new = np.concatenate([new, chunk])
    return ctx.astype(np.int64), new.astype(np.int64)


def _read_lens(case, ctx, new):
    """How many of each sequence's last tokens are read back: everything, or (after an append) the
    rows of the blocks it touched."""
    if case["op"] == "read":
        return ctx
    first = (ctx - new) // case["bs"] * case["bs"]
    return ctx - first


def _padded(case):
    """Values of the largest padded tensor of the plain form."""
    ctx, new = _lens(case)
    if case["op"] != "attention":
        return float(_read_lens(case, ctx, new).sum() * case["hkv"] * case["d"])
    one, many = new == 1, new > 1
    size = 0.0
    for m in (one, many):
        if m.any():
            size = max(size, float(m.sum() * ctx[m].max() * max(case["hkv"] * case["d"], case["hq"] * new[m].max())))
    return size


def work(case):
    ctx, new = _lens(case)
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    T = int(new.sum())
    row = hkv * d
    tables = 4.0 * (-(-ctx // bs)).sum()
    if case["op"] == "attention":
        keys = float(ctx.sum())
        scales = 8.0 * hkv * (-(-ctx // bs)).sum()
        pairs = float((new * ctx - new * (new - 1) // 2).sum())  # (query, visible key) pairs
        return {"bytes": 2.0 * keys * row + scales + tables + 4.0 * T * hq * d, "flops": 4.0 * pairs * hq * d}
    back = float(_read_lens(case, ctx, new).sum())
    blocks = float((-(-_read_lens(case, ctx, new) // bs)).sum())
    read = 2.0 * back * row * (1 + 2) + 8.0 * hkv * blocks + 4.0 * blocks
    if case["op"] == "read":
        return {"bytes": read, "flops": 2.0 * back * row}
    # append: q read and written, k and v read, both written in 8 bits; then the read back
    append = 4.0 * T * hq * d + 4.0 * T * row + 2.0 * T * row + 8.0 * hkv * blocks + 4.0 * blocks
    return {"bytes": append + read, "flops": 3.0 * T * (hq + hkv) * d + 4.0 * T * row + 2.0 * back * row}


# ------------------------------------------------------------------------------ the inputs


def _exponent(amax, dtype):
    """The smallest e >= -100 with amax <= LARGEST * 2^e, amax float32 or float64."""
    m, x = torch.frexp(amax)  # amax = m 2^x, m in [0.5, 1)
    e = x - 7 + (m > 127.0 / 128) if dtype == "int8" else x - 9 + (m > 0.875)
    return torch.where(amax > 0, e, torch.full_like(e, -100)).clamp(min=-100)


def _two_to(e):
    """2^e in float32, exactly (torch.ldexp and exp2 go through a rounded power)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _hold(x, dtype):
    """x already divided by its scale, as the type holds it."""
    if dtype == "int8":
        return torch.round(x).clamp(-127, 127).to(torch.int8)
    return x.float().clamp(-448, 448).to(torch.float8_e4m3fn)


def _values(g, shape, channel):
    """Normal values whose tokens and channels differ in size, as keys and values do."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= torch.exp(0.4 * torch.randn(shape[:-1] + (1,), generator=g, device="cuda"))
    return (x * channel).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ctx, new = _lens(case)
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    blocks = -(-ctx // bs)
    num_blocks = int(blocks.sum() + blocks.sum() // 8 + 3)
    order = torch.randperm(num_blocks, generator=g, device="cuda").to(torch.int32)
    held = np.arange(int(blocks.max()))[None, :] < blocks[:, None]
    at = np.where(held, np.cumsum(held.reshape(-1)).reshape(held.shape) - 1, 0)
    held = torch.from_numpy(held).cuda()
    tables = torch.where(held, order[torch.from_numpy(at).cuda()], torch.full_like(order[:1], -1))
    channel = torch.exp(0.6 * torch.randn(2, 1, hkv, d, generator=g, device="cuda"))
    s = {"case": dict(case), "tables": tables, "scale": d ** -0.5,
         "ctx": torch.from_numpy(ctx.astype(np.int32)).cuda(),
         "qsl": torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()}
    for i, name in enumerate("kv"):
        cache = torch.empty(num_blocks, bs, hkv, d, dtype=DTYPES[case["dtype"]], device="cuda")
        scale = torch.empty(num_blocks, hkv, device="cuda")
        step = max(1, (1 << 26) // (bs * hkv * d))
        for b in range(0, num_blocks, step):  # a part of the pool at a time
            x = _values(g, (min(step, num_blocks - b), bs, hkv, d), channel[i]).float()
            e = _exponent(x.abs().amax(dim=(1, 3)), case["dtype"])
            scale[b:b + step] = _two_to(e)
            cache[b:b + step] = _hold(x * _two_to(-e[:, None, :, None]), case["dtype"])
        s[name + "_cache"], s[name + "_scale"] = cache, scale
    T = int(new.sum())
    if case["op"] != "read":
        s["q"] = torch.randn(T, hq, d, generator=g, device="cuda").to(torch.bfloat16)
    if case["op"] == "append":
        s["q_rot"] = torch.empty_like(s["q"])
        s["k"] = _values(g, (T, hkv, d), channel[0])
        s["v"] = _values(g, (T, hkv, d), channel[1])
    if case["op"] == "attention":
        s["out"] = torch.empty_like(s["q"])
        # how the plain form pads its queries and keys: the step's sequences by kind
        kinds = [np.flatnonzero(new == 1), np.flatnonzero(new > 1)]
        s["kinds"] = [(torch.from_numpy(k).cuda(), int(ctx[k].max()), int(new[k].max())) for k in kinds if k.size]
    else:
        rows = _read_lens(case, ctx, new)
        s["rsl"] = torch.from_numpy(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)).cuda()
        s["k_out"] = torch.empty(int(rows.sum()), hkv, d, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.empty_like(s["k_out"])
    return s


# --------------------------------------------------------------------------- the plain form


def _tokens(start, ctx, count):
    """Sequence and position of each of the `count` rows that `start` hands out."""
    t = torch.arange(count, device="cuda")
    b = torch.searchsorted(start.long(), t, right=True) - 1
    return b, ctx.long()[b] - start.long()[b + 1] + t


def _plain_rope(x, pos):
    half = x.shape[-1] // 2
    f = THETA ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    a = (pos.double()[:, None] * f)[:, None, :]
    lo, hi = x[..., :half].double(), x[..., half:].double()
    return torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1).float()


def _plain_quantise(s, x, cache, scale):
    """x [T, Hkv, d] float32 into its slots: one scale for each block and head."""
    c, bs = s["case"], s["case"]["bs"]
    b, pos = _tokens(s["qsl"], s["ctx"], x.shape[0])
    block = s["tables"].long()[b, pos // bs]
    amax = torch.zeros_like(scale).scatter_reduce(0, block[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
    # only a sequence's first block of the step can hold rows already
    first_pos = s["ctx"].long() - (s["qsl"][1:] - s["qsl"][:-1]).long()
    first = s["tables"].long().gather(1, (first_pos // bs)[:, None])[:, 0]
    before = (first_pos % bs)[:, None]
    e_old = torch.frexp(scale[first])[1] - 1
    e = _exponent(amax, c["dtype"])
    e[first] = torch.where(before > 0, torch.maximum(e[first], e_old), e[first])
    down = torch.where(before > 0, e[first] - e_old, torch.zeros_like(e_old))
    raw = cache.view(torch.int8)  # (indexing by the bytes: the same for either type)
    old = raw[first]
    moved = _hold(old.view(cache.dtype).float() * _two_to(-down[:, None, :, None]), c["dtype"]).view(torch.int8)
    there = torch.arange(bs, device="cuda")[None, :] < before
    raw[first] = torch.where(there[:, :, None, None], moved, old)
    raw[block, pos % bs] = _hold(x * _two_to(-e[block])[:, :, None], c["dtype"]).view(torch.int8)
    scale[block] = _two_to(e[block])


def _plain_append(s):
    pos = _tokens(s["qsl"], s["ctx"], s["q"].shape[0])[1]
    _plain_quantise(s, _plain_rope(s["k"], pos), s["k_cache"], s["k_scale"])
    _plain_quantise(s, s["v"].float(), s["v_cache"], s["v_scale"])
    return _plain_rope(s["q"], pos).to(torch.bfloat16)


def _plain_read(s, cache, scale):
    bs = s["case"]["bs"]
    b, pos = _tokens(s["rsl"], s["ctx"], s["k_out"].shape[0])
    block = s["tables"].long()[b, pos // bs]
    held = cache.view(torch.int8)[block, pos % bs].view(cache.dtype)
    return (held.float() * scale[block][:, :, None]).to(torch.bfloat16)


def _plain_padded(cache, scale, table):
    """The blocks of `table` [S, n] as one row of float32 tokens for each sequence."""
    held = cache.view(torch.int8)[table].view(cache.dtype).float()
    return (held * scale[table][:, :, None, :, None]).flatten(1, 2)


def _plain_kind(s, out, seqs, keys, rows):
    """Attention of the sequences `seqs`, keys padded to `keys` and queries to `rows`."""
    c, T = s["case"], s["q"].shape[0]
    bs, hq, hkv, d = c["bs"], c["hq"], c["hkv"], c["d"]
    S, G = seqs.shape[0], hq // hkv
    ctx, start, end = s["ctx"].long()[seqs], s["qsl"].long()[seqs], s["qsl"].long()[seqs + 1]
    blocks = -(-keys // bs)
    table = s["tables"][seqs, :blocks].long().clamp(min=0)
    k, v = (_plain_padded(s[n + "_cache"], s[n + "_scale"], table).transpose(1, 2) for n in "kv")
    r = torch.arange(rows, device="cuda")[None, :]
    row = torch.where(start[:, None] + r < end[:, None], start[:, None] + r, torch.full_like(r, T))  # T: a spare row
    pos = ctx[:, None] - (end - start)[:, None] + r
    q = s["q"][row.clamp(max=T - 1)].float().view(S, rows, hkv, G, d)
    q = q.permute(0, 2, 3, 1, 4).reshape(S, hkv, G * rows, d)
    p = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(S, hkv, G, rows, -1)
    seen = torch.arange(blocks * bs, device="cuda") <= pos[:, :, None]
    p.masked_fill_(~seen[:, None, None], -math.inf)
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(p.view(S, hkv, G * rows, -1), v).view(S, hkv, G, rows, d) / p.sum(-1, keepdim=True)
    out[row.reshape(-1)] = o.permute(0, 3, 1, 2, 4).reshape(S * rows, hq, d)


def _plain_attention(s):
    out = torch.empty(s["q"].shape[0] + 1, *s["q"].shape[1:], device="cuda")
    [_plain_kind(s, out, *kind) for kind in s["kinds"]]
    return out[:-1].to(torch.bfloat16)


# ------------------------------------------------------------------------ this package's calls


def _own_read(s):
    from paged_kv_gqa_14_gb300 import ops

    ops.kv_read_q8(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["tables"], s["ctx"], s["rsl"],
                   s["k_out"], s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _own_append(s):
    from paged_kv_gqa_14_gb300 import ops

    s["q_rot"].copy_(s["q"])  # the call rotates q in place; a step's q is new, this one is used again
    ops.kv_append_q8(s["q_rot"], s["k"], s["v"], s["tables"], s["ctx"], s["qsl"], s["k_cache"], s["v_cache"],
                     s["k_scale"], s["v_scale"], THETA)
    return {"q": s["q_rot"], **_own_read(s)}


def _own_attention(s):
    from paged_kv_gqa_14_gb300 import ops

    if "workspace" not in s:  # allocated once, as an engine does
        T, hq, d = s["q"].shape
        s["workspace"] = ops.alloc_workspace(T, s["ctx"].shape[0], hq, s["case"]["hkv"], d, s["tables"].shape[1])
    ops.paged_attention_q8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["tables"], s["ctx"],
                           s["qsl"], s["scale"], out=s["out"], workspace=s["workspace"])
    return {"out": s["out"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "read": _own_read, "attention": _own_attention}[op](state)
    if op == "attention":
        return {"out": _plain_attention(state)}
    q = {"q": _plain_append(state)} if op == "append" else {}
    return {**q, "k": _plain_read(state, state["k_cache"], state["k_scale"]),
            "v": _plain_read(state, state["v_cache"], state["v_scale"])}


# ------------------------------------------------------------------ the definition in 64 bits


def _turned(x, positions):
    """x [n, heads, d] float64 with each pair (i, i + d/2) turned by position * theta^(-2i/d)."""
    d = x.shape[2]
    out = torch.empty_like(x)
    for i in range(d // 2):
        angle = positions * THETA ** (-2.0 * i / d)
        cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        out[:, :, i] = x[:, :, i] * cos - x[:, :, i + d // 2] * sin
        out[:, :, i + d // 2] = x[:, :, i + d // 2] * cos + x[:, :, i] * sin
    return out


def _on_grid(x, step, dtype):
    """Float64 values rounded to what the type holds with this scale (ties to even)."""
    y = x / step
    if dtype == "int8":
        return torch.round(y).clamp(-127, 127) * step
    # three bits behind the point, 2^-9 at least: y in [2^(n-1), 2^n) has steps of 2^(n-4)
    ulp = (torch.frexp(y)[1].clamp(min=-5).long() - 4 + 1023 << 52).view(torch.float64)
    return (torch.round(y / ulp) * ulp).clamp(-448, 448) * step


def exact(case, seed):
    s = prepare(case, seed)
    ctx, new = _lens(case)
    bs, hq, hkv, d, kind = case["bs"], case["hq"], case["hkv"], case["d"], case["dtype"]
    tables = s["tables"].cpu().numpy()
    starts = np.concatenate([[0], np.cumsum(new)])

    def contiguous(name, b, lo, hi):
        """Keys or values of sequence b at positions lo .. hi - 1, with their scales."""
        p = np.arange(lo, hi)
        block = torch.from_numpy(tables[b, p // bs].astype(np.int64)).cuda()
        row = torch.from_numpy(p % bs).cuda()
        cache = s[name + "_cache"]
        held = cache.view(torch.int8)[block, row].view(cache.dtype)
        return held.to(torch.float32).double(), s[name + "_scale"][block].double()

    if case["op"] == "read":
        return {n: torch.cat([torch.mul(*(lambda x, e: (x, e[:, :, None]))(*contiguous(n, b, 0, int(ctx[b]))))
                              for b in range(len(ctx))]) for n in "kv"}
    if case["op"] == "append":
        got = {"q": [], "k": [], "v": []}
        for b in range(len(ctx)):
            t0, t1 = int(starts[b]), int(starts[b + 1])
            first = int(ctx[b] - new[b])
            pos = torch.arange(first, int(ctx[b]), device="cuda", dtype=torch.float64)
            got["q"].append(_turned(s["q"][t0:t1].double(), pos))
            for n in "kv":
                x = s[n][t0:t1].double()
                x = _turned(x, pos) if n == "k" else x
                base = first // bs * bs
                for lo in range(base, int(ctx[b]), bs):
                    hi = min(lo + bs, int(ctx[b]))
                    fresh = x[max(0, lo - first):hi - first]
                    need = fresh.abs().amax(dim=(0, 2)).clamp(min=1e-40) / LARGEST[kind]
                    m, x2 = torch.frexp(need)
                    up = torch.where(m == 0.5, x2 - 1, x2).clamp(min=-100).long()  # the least with need <= 2^up
                    step = (up + 1023 << 52).view(torch.float64)
                    rows = []
                    if lo < first:  # rows that were there: rounded again where the scale grows
                        old, was = contiguous(n, b, lo, first)
                        step = torch.maximum(step, was[0])
                        rows.append(_on_grid(old * was[:, :, None], step[None, :, None], kind))
                    rows.append(_on_grid(fresh, step[None, :, None], kind))
                    got[n] += rows
        return {n: torch.cat(got[n]) for n in got}
    if work(case)["flops"] > 1e12:
        return None
    out = torch.empty(int(new.sum()), hq, d, dtype=torch.float64, device="cuda")
    for b in range(len(ctx)):
        k, ke = contiguous("k", b, 0, int(ctx[b]))
        v, ve = contiguous("v", b, 0, int(ctx[b]))
        limit = torch.arange(int(ctx[b] - new[b]), int(ctx[b]), device="cuda")
        late = torch.arange(int(ctx[b]), device="cuda")[None, :] > limit[:, None]
        for h in range(hkv):
            kh, vh = k[:, h] * ke[:, h, None], v[:, h] * ve[:, h, None]
            heads = range(h * (hq // hkv), (h + 1) * (hq // hkv))
            if new[b] == 1:
                w = torch.softmax(s["q"][starts[b], heads.start:heads.stop].double() @ kh.T * s["scale"], -1)
                out[starts[b], heads.start:heads.stop] = w @ vh
                continue
            for i in heads:
                score = s["q"][starts[b]:starts[b + 1], i].double() @ kh.T * s["scale"]
                out[starts[b]:starts[b + 1], i] = torch.softmax(score.masked_fill(late, -math.inf), -1) @ vh
    return {"out": out}
