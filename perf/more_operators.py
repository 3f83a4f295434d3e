"""Attention variants over the paged bf16 cache as they are measured: cases, inputs, a plain form in torch and
the calls of this package.

k_cache and v_cache are [num_blocks, block_size, Hkv, d] bfloat16; sequence b owns query rows
query_start_loc[b] : query_start_loc[b + 1] and context_lens[b] keys, its rows being the last tokens of them.

  diff  differential attention.  Head h of Hq / 2 uses q heads 2h and 2h + 1; with g = h // (Hq / Hkv) they attend to
        k heads 2g and 2g + 1, and the values are v heads 2g and 2g + 1 side by side (2d numbers):
            x = softmax(scale q_2h K_2g) V - lam_h softmax(scale q_2h+1 K_2g+1) V
            out = out_scale x                                    without a norm weight
            out = out_scale weight x / sqrt(mean(x^2) + eps)     with one
        lam is one number for each head, or for each token and head.
  bias  attention with a learned relative position bias: the key at distance n = position - key's position adds
        bias[bucket(n), head] to its score.  Half of the buckets hold one distance each, the others grow
        logarithmically up to max_distance, beyond which all distances share the last.

Both take decode tokens and causal prefill chunks in one call.
"""

import math

import numpy as np
import torch

own = False

EPS = 1.0e-5


def _case(op, hq, hkv, d, bs, dec=0, lo=1, hi=1, pre=0, chunk=0, prior=0, lens=0, lam="head", norm=True, buckets=32,
          far=128, table="fp32"):
    """dec sequences of one new token with contexts in [lo, hi]; pre sequences with chunks of up to `chunk` new
    tokens behind up to `prior` cached ones; `lens` seeds the lengths.  lam and norm are for diff, buckets, far
    (max_distance) and table (the bias table's type) for bias."""
    c = {"op": op, "hq": hq, "hkv": hkv, "d": d, "bs": bs, "dec": dec, "lo": lo, "hi": hi, "pre": pre, "chunk": chunk,
         "prior": prior, "lens": lens}
    return {**c, **({"lam": lam, "norm": norm} if op == "diff" else {"buckets": buckets, "far": far, "table": table})}


def listed():
    cases = {
        # the smallest call: four short contexts
        "diff-4": _case("diff", 4, 2, 64, 16, dec=4, lo=1, hi=100, lens=1, norm=False),
        # a small decode batch, head_dim 64, a group of seven, lam from the token
        "diff-32": _case("diff", 14, 2, 64, 16, dec=32, lo=129, hi=1152, lens=2, lam="token"),
        # 256 decode sequences of up to 2048 tokens: an ordinary serving step
        "diff-256": _case("diff", 16, 8, 128, 16, dec=256, lo=100, hi=2048, lens=3),
        # one user with a very long context: the split over the keys alone fills the GPU
        "diff-1x128k": _case("diff", 32, 8, 128, 64, dec=1, lo=131000, hi=131072, lens=4),
        # a mixed step: 200 decode tokens beside four prefill chunks
        "diff-mixed": _case("diff", 16, 8, 128, 16, dec=200, lo=64, hi=2048, pre=4, chunk=512, prior=1536, lens=5),
        # a long prompt's late chunk: compute alone
        "diff-chunk-16k": _case("diff", 28, 4, 128, 32, pre=1, chunk=4096, prior=12288, lens=6),
        # the smallest call
        "bias-4": _case("bias", 4, 2, 64, 16, dec=4, lo=1, hi=100, lens=7),
        # an ordinary serving step, the table in the model's own type
        "bias-256": _case("bias", 16, 8, 128, 16, dec=256, lo=100, hi=2048, lens=8, table="bf16"),
        # long contexts, a group of seven, buckets that reach far back
        "bias-50x8k": _case("bias", 28, 4, 128, 32, dec=50, lo=8000, hi=8192, lens=9, buckets=64, far=2048),
        # a mixed step
        "bias-mixed": _case("bias", 16, 8, 128, 16, dec=200, lo=64, hi=2048, pre=4, chunk=512, prior=1536, lens=10),
        # a budget of 8192 tokens of fresh prompts, head_dim 64: a third of the scores near the diagonal
        "bias-prompts": _case("bias", 14, 2, 64, 16, pre=5, chunk=2048, prior=700, lens=11),
        # a long prompt's late chunk
        "bias-chunk-16k": _case("bias", 28, 4, 128, 32, pre=1, chunk=4096, prior=12288, lens=12, table="bf16"),
    }
    return [dict(c, name=n) for n, c in cases.items()]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["diff", "bias"])
        hkv = rng.choice([2, 4, 8] if op == "diff" else [1, 2, 4, 8])
        c = _case(op, hkv * rng.randint(1, 8), hkv, rng.choice([64, 128]), rng.choice([8, 16, 32, 64, 128]),
                  lens=rng.randint(100, 10**6), lam=rng.choice(["head", "token"]), norm=rng.random() < 0.7,
                  buckets=rng.choice([8, 32, 64, 128]), table=rng.choice(["fp32", "bf16"]))
        if op == "bias":
            c["far"] = c["buckets"] * rng.choice([1, 4, 16]) + rng.randint(0, 40)
        kind = rng.choice(["dec", "dec", "pre", "mixed"])
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
    """Context lengths (with the step's new tokens) and new tokens of each sequence, decode sequences first; part
    of the case, whatever the seed of the values."""
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


def _padded(case):
    """Values of the largest padded tensor of the plain form."""
    ctx, new = _lens(case)
    one, many = new == 1, new > 1
    size = 0.0
    for m in (one, many):
        if m.any():
            size = max(size, float(m.sum() * ctx[m].max() * max(case["hkv"] * case["d"], case["hq"] * new[m].max())))
    return size


def work(case):
    ctx, new = _lens(case)
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    T = float(new.sum())
    pairs = float((new * ctx - new * (new - 1) // 2).sum())  # (query, visible key) pairs
    moved = 4.0 * float(ctx.sum()) * hkv * d + 4.0 * float((-(-ctx // bs)).sum()) + 4.0 * T * hq * d
    if case["op"] == "diff":
        lam = 2.0 * hq * (T if case["lam"] == "token" else 1.0)
        return {"bytes": moved + lam + (8.0 * d if case["norm"] else 0.0), "flops": 6.0 * pairs * hq * d}
    return {"bytes": moved + (4.0 if case["table"] == "fp32" else 2.0) * case["buckets"] * hq,
            "flops": 4.0 * pairs * hq * d}


# ------------------------------------------------------------------------------ the inputs


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
        cache = torch.empty(num_blocks, bs, hkv, d, dtype=torch.bfloat16, device="cuda")
        step = max(1, (1 << 26) // (bs * hkv * d))
        for b in range(0, num_blocks, step):  # a part of the pool at a time
            cache[b:b + step] = _values(g, (min(step, num_blocks - b), bs, hkv, d), channel[i])
        s[name + "_cache"] = cache
    T = int(new.sum())
    s["q"] = torch.randn(T, hq, d, generator=g, device="cuda").to(torch.bfloat16)
    if case["op"] == "diff":
        shape = (T, hq // 2) if case["lam"] == "token" else (hq // 2,)
        s["lam"] = 0.2 + 0.6 * torch.rand(shape, generator=g, device="cuda")
        s["weight"] = 1.0 + 0.2 * torch.randn(2 * d, generator=g, device="cuda") if case["norm"] else None
        s["out_scale"] = 0.2 + 0.6 * float(torch.rand((), generator=g, device="cuda"))
        s["out"] = torch.empty(T, hq // 2, 2 * d, dtype=torch.bfloat16, device="cuda")
    else:
        s["starts"] = torch.tensor(_starts(case["buckets"], case["far"]), device="cuda")
        bias = torch.randn(case["buckets"], hq, generator=g, device="cuda")
        s["bias"] = bias if case["table"] == "fp32" else bias.to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
    # how the plain form pads its queries and keys: the step's sequences by kind
    kinds = [np.flatnonzero(new == 1), np.flatnonzero(new > 1)]
    s["kinds"] = [(torch.from_numpy(k).cuda(), int(ctx[k].max()), int(new[k].max())) for k in kinds if k.size]
    return s


# --------------------------------------------------------------------------- the plain form


def _starts(buckets, far):
    """The least distance of each bucket, in whole numbers: bucket e + j starts at the least n with
    (n / e)^k >= (far / e)^j, e single distances and k = buckets - e."""
    e = buckets // 2
    k = buckets - e
    starts, n = list(range(e)), e
    for j in range(k):
        while n ** k < far ** j * e ** (k - j):
            n += 1
        starts.append(n)
    return starts


def _plain_kind(s, out, seqs, keys, rows):
    """Attention of the sequences `seqs`, keys padded to `keys` and queries to `rows`."""
    c, T = s["case"], s["q"].shape[0]
    bs, hq, hkv, d = c["bs"], c["hq"], c["hkv"], c["d"]
    S, G, diff = seqs.shape[0], hq // hkv, c["op"] == "diff"
    ctx, start, end = s["ctx"].long()[seqs], s["qsl"].long()[seqs], s["qsl"].long()[seqs + 1]
    blocks = -(-keys // bs)
    table = s["tables"][seqs, :blocks].long().clamp(min=0)
    k, v = (s[n + "_cache"][table].float().flatten(1, 2).transpose(1, 2) for n in "kv")  # [S, Hkv, keys, d]
    r = torch.arange(rows, device="cuda")[None, :]
    row = torch.where(start[:, None] + r < end[:, None], start[:, None] + r, torch.full_like(r, T))  # T: a spare row
    pos = ctx[:, None] - (end - start)[:, None] + r
    distance = pos[:, :, None] - torch.arange(blocks * bs, device="cuda")  # [S, rows, keys]
    q = s["q"][row.clamp(max=T - 1)].float()  # [S, rows, Hq, d]

    def weights(q, k, bias):
        """Softmax of q [S, rows, h, d] over k [S, h / G, keys, d], and 1 / its sum."""
        q = q.reshape(S, rows, -1, G, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
        p = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(S, -1, G, rows, blocks * bs)
        if bias is not None:
            p.add_(bias)
        p.masked_fill_((distance < 0)[:, None, None], -math.inf)
        p.sub_(p.amax(-1, keepdim=True)).exp_()
        return p.view(S, -1, G * rows, blocks * bs), p.sum(-1, keepdim=True)

    if not diff:
        bucket = torch.bucketize(distance.clamp(min=0), s["starts"], right=True) - 1
        bias = torch.empty(S, hkv, G, rows, blocks * bs, device="cuda")
        for h in range(hq):
            bias[:, h // G, h % G] = s["bias"].float()[:, h][bucket]
        p, total = weights(q, k, bias)
        o = torch.matmul(p, v).view(S, hkv, G, rows, d) / total
        out[row.reshape(-1)] = o.permute(0, 3, 1, 2, 4).reshape(S * rows, hq, d)
        return
    v = torch.cat([v[:, 0::2], v[:, 1::2]], -1)  # [S, Hkv / 2, keys, 2d]
    maps = []
    for part in (0, 1):
        p, total = weights(q[:, :, part::2], k[:, part::2], None)
        maps.append((torch.matmul(p, v).view(S, -1, G, rows, 2 * d) / total).permute(0, 3, 1, 2, 4).flatten(2, 3))
        del p
    lam = s["lam"] if c["lam"] == "head" else s["lam"][row.clamp(max=T - 1)]
    x = maps[0] - lam[..., None] * maps[1]  # [S, rows, Hq / 2, 2d]
    if c["norm"]:
        x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["weight"]
    out[row.reshape(-1)] = (x * s["out_scale"]).flatten(0, 1)


def _plain(s):
    out = torch.empty(s["q"].shape[0] + 1, *s["out"].shape[1:], device="cuda")
    [_plain_kind(s, out, *kind) for kind in s["kinds"]]
    return out[:-1].to(torch.bfloat16)


# ------------------------------------------------------------------------ this package's calls


def _own(s):
    from paged_kv_gqa_14_gb300 import ops

    c = s["case"]
    diff = c["op"] == "diff"
    if "workspace" not in s:  # allocated once, as an engine does
        T, hq, d = s["q"].shape
        s["workspace"] = ops.alloc_workspace(T, s["ctx"].shape[0], hq, c["hkv"], d, s["tables"].shape[1], diff=diff)
        if not diff:
            s["buckets"] = ops.relative_buckets(c["buckets"], c["far"])
    call = (s["q"], s["k_cache"], s["v_cache"], s["tables"], s["ctx"], s["qsl"], s["scale"])
    if diff:
        return ops.paged_attention_diff(*call, s["lam"], norm_weight=s["weight"], norm_eps=EPS,
                                        out_scale=s["out_scale"], out=s["out"], workspace=s["workspace"])
    return ops.paged_attention_bias(*call, s["bias"], s["buckets"], out=s["out"], workspace=s["workspace"])


def run(state):
    return {"out": _own(state) if own else _plain(state)}


# ------------------------------------------------------------------ the definition in 64 bits


def _bucket_of(n, buckets, far):
    """Bucket of one distance by its formula, the floor of a logarithm's ratio found with whole numbers."""
    exact_ones = buckets // 2
    if n < exact_ones:
        return n
    rest, j = buckets - exact_ones, 0
    # floor(rest log(n / e) / log(far / e)) is the largest j with (far / e)^j <= (n / e)^rest
    while j < rest - 1 and far ** (j + 1) * exact_ones ** (rest - j - 1) <= n ** rest:
        j += 1
    return exact_ones + j


def exact(case, seed):
    if work(case)["flops"] > 2e12:
        return None
    s = prepare(case, seed)
    ctx, new = _lens(case)
    bs, hq, hkv, d = case["bs"], case["hq"], case["hkv"], case["d"]
    tables = s["tables"].cpu().numpy()
    starts = np.concatenate([[0], np.cumsum(new)])
    diff, G = case["op"] == "diff", hq // hkv
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    if not diff:
        by_distance = torch.tensor([_bucket_of(n, case["buckets"], case["far"]) for n in range(case["far"] + 1)],
                                   device="cuda")
        bias = s["bias"].double()
    for b in range(len(ctx)):
        t0, t1, keys = int(starts[b]), int(starts[b + 1]), int(ctx[b])
        p = np.arange(keys)
        block = torch.from_numpy(tables[b, p // bs].astype(np.int64)).cuda()
        at = torch.from_numpy(p % bs).cuda()
        k, v = s["k_cache"][block, at], s["v_cache"][block, at]
        position = torch.arange(keys - int(new[b]), keys, device="cuda")
        back = position[:, None] - torch.arange(keys, device="cuda")[None, :]

        def attend(i, kh, values):
            score = s["q"][t0:t1, i].double() @ k[:, kh].double().T * s["scale"]
            if not diff:
                score += bias[:, i][by_distance[back.clamp(0, case["far"])]]
            return torch.softmax(score.masked_fill_(back < 0, -math.inf), -1) @ values

        for h in range(hq // 2 if diff else hq):
            if not diff:
                out[t0:t1, h] = attend(h, h // G, v[:, h // G].double())
                continue
            g = h // G
            both = torch.cat([v[:, 2 * g], v[:, 2 * g + 1]], -1).double()
            lam = (s["lam"][t0:t1, h, None] if case["lam"] == "token" else s["lam"][h]).double()
            x = attend(2 * h, 2 * g, both) - lam * attend(2 * h + 1, 2 * g + 1, both)
            if case["norm"]:
                x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"].double()
            out[t0:t1, h] = x * s["out_scale"]
    return {"out": out}
