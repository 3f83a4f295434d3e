"""Helpers for the tests of the attention variants: seeded batches over a poisoned pool, the calls and their oracle.
Outputs have to lie within the oracle's slack, which is derived there from the roundings that a call may make."""

import numpy as np
import torch

import oracle
from oracle import variants as OV
from paged_kv_gqa_14_gb300 import ops
from paged_kv_gqa_14_gb300 import workloads as W
from tests.gpu_util import bf16_to_dev, idx_to_dev

FLOOR = 1e-6  # absolute, where an output is 0


class Batch:
    """A step after its append, on the host and on the GPU; rows of the pool that hold no key are NaN."""

    def __init__(self, ctx, spans, hq, hkv, d, bs=16, seed=0, extra_tokens=0, gain=1.0, scale=None):
        ctx, spans = np.asarray(ctx), np.asarray(spans)
        nb = int((-(-ctx // bs)).sum()) + 4
        bt = W.make_batch(ctx, spans, hq, hkv, d, nb, seed=seed, block_size=bs)
        q, kc, vc = oracle.kv_append(bt.q, bt.k, bt.v, bt.positions, bt.slot_mapping, bt.k_cache, bt.v_cache,
                                     bt.rope_theta)
        if gain != 1.0:
            q = oracle.f64_to_bf16_bits(oracle.bf16_bits_to_f64(q) * gain)
        if extra_tokens:  # rows behind the last sequence
            q = np.concatenate([q, W.normal_bf16(np.random.default_rng(seed + 1), (extra_tokens, hq, d))])
        self.bt, self.q, self.kc, self.vc = bt, q, kc, vc
        self.scale = float(d**-0.5) if scale is None else scale
        self.d, self.hq, self.hkv, self.T = d, hq, hkv, q.shape[0]

    def host(self):
        b = self.bt
        return self.q, self.kc, self.vc, b.block_tables, b.context_lens, b.query_start_loc, self.scale

    def dev(self):
        b = self.bt
        return (bf16_to_dev(self.q), bf16_to_dev(self.kc), bf16_to_dev(self.vc), idx_to_dev(b.block_tables),
                idx_to_dev(b.context_lens), idx_to_dev(b.query_start_loc), self.scale)


def lam_of(batch, seed, per_token=False):
    rng = np.random.default_rng(seed)
    shape = (batch.T, batch.hq // 2) if per_token else (batch.hq // 2,)
    return rng.uniform(0.2, 0.8, shape).astype(np.float32)


def weight_of(batch, seed):
    return np.random.default_rng(seed).normal(1.0, 0.2, 2 * batch.d).astype(np.float32)


def bias_of(batch, num_buckets, seed, bf16=False):
    """(what the call gets, its values in 64 bits)"""
    x = torch.from_numpy(np.random.default_rng(seed).normal(0.0, 1.0, (num_buckets, batch.hq)).astype(np.float32))
    x = x.to(torch.bfloat16) if bf16 else x
    return x, x.double().numpy()


def within(got, ref, slack, what=""):
    """Every number in its slack, rows that no span covers left as they were (marked 7 before the call)."""
    got = got.double().cpu().numpy()
    free = np.isnan(ref)
    assert np.all(got[free] == 7.0), f"{what}: a row outside every span was written"
    got, ref, slack = got[~free], ref[~free], slack[~free]
    assert np.all(np.isfinite(got)), f"{what}: {np.count_nonzero(~np.isfinite(got))} outputs are not finite"
    over = np.abs(got - ref) / (slack + FLOOR)
    at = int(over.argmax()) if over.size else 0
    assert over.size == 0 or over[at] <= 1.0, (
        f"{what}: {np.count_nonzero(over > 1)} of {over.size} past their slack, worst {got[at]} for {ref[at]} "
        f"({over[at]:.2f} of {slack[at]:.2e})")
    return float(over.max()) if over.size else 0.0


def marked(*shape):
    return torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")


def check_bias(batch, buckets, bias, bias64, starts, what="", **kw):
    ref, slack = OV.paged_attention_bias(*batch.host(), bias64, starts)
    out = marked(batch.T, batch.hq, batch.d)
    got = ops.paged_attention_bias(*batch.dev(), bias.cuda(), buckets, out=out, **kw)
    torch.cuda.synchronize()
    assert got is out and ops.get_device_error() == 0
    return within(out, ref, slack, what)


def check_diff(batch, lam, weight=None, eps=1e-5, out_scale=1.0, what="", **kw):
    ref, slack = OV.paged_attention_diff(*batch.host(), lam, weight, eps, out_scale)
    out = marked(batch.T, batch.hq // 2, 2 * batch.d)
    got = ops.paged_attention_diff(*batch.dev(), torch.from_numpy(lam).cuda(),
                                   norm_weight=None if weight is None else torch.from_numpy(weight).cuda(),
                                   norm_eps=eps, out_scale=out_scale, out=out, **kw)
    torch.cuda.synchronize()
    assert got is out and ops.get_device_error() == 0
    return within(out, ref, slack, what)
