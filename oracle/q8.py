"""The 8-bit KV cache in fp64 (test infrastructure only): what its bytes stand for, the quantised
append, and which roundings an fp32 rotation may take either way.

Format: a pool of bytes [num_blocks, block_size, Hkv, d], "int8" (two's complement, written values
within 127) or "e4m3" (fp8, written values within 448), and one power-of-two scale for each block and
kv head; a held value x stands for x * scale.

Append: the new rows of a block share the smallest power of two (2^-100 at least) with which their
largest finite magnitude fits, and at least the block's present scale when rows before them are there;
those are rounded to a scale that grew.
"""

import numpy as np

from .bf16 import bf16_bits_to_f64, f64_to_bf16_bits
from .rope import rope64

LARGEST = {"int8": 127.0, "e4m3": 448.0}
MIN_SCALE = 2.0**-100


def e4m3_values():
    """The value of each of the 256 e4m3 codes: sign, four exponent bits (bias 7), three fraction
    bits; exponent 0 is subnormal, 0x7f and 0xff are NaN, there are no infinities."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, f * 2.0**-9, (8 + f) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def decode(codes, kind):
    """Bytes to the fp64 values they hold."""
    codes = np.asarray(codes, dtype=np.uint8)
    return codes.view(np.int8).astype(np.float64) if kind == "int8" else e4m3_values()[codes]


def encode(x, kind):
    """fp64 values to the nearest held ones (ties to even), as bytes; infinities to the largest, NaN
    to 0 (int8) or NaN (e4m3)."""
    x = np.asarray(x, dtype=np.float64)
    if kind == "int8":
        return np.where(np.isnan(x), 0.0, np.clip(np.rint(x), -127, 127)).astype(np.int8).view(np.uint8)
    grid = e4m3_values()[:127]
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    hi = np.clip(np.searchsorted(grid, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    below, above = a - grid[lo], grid[hi] - a
    code = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(x), 127, code)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def scale_for(amax, kind):
    """The smallest power of two, 2^-100 at least, with amax <= LARGEST * scale."""
    m, x = np.frexp(np.asarray(amax, dtype=np.float64) / LARGEST[kind])
    return np.maximum(np.ldexp(1.0, np.where(m == 0.5, x - 1, np.where(m == 0, -200, x))), MIN_SCALE)


def dequantise(codes, scale, kind):
    """The bf16 bit patterns the whole pool stands for (exact for finite values)."""
    return f64_to_bf16_bits(decode(codes, kind) * np.asarray(scale, np.float64)[:, None, :, None])


def kv_append_q8(q, k, v, block_tables, context_lens, query_start_loc, k_cache, v_cache, k_scale, v_scale,
                 rope_theta, kind):
    """Returns (q_rot bits, k_cache, v_cache, k_scale, v_scale, k_exact): copies with the step's tokens
    written; k_exact holds the unrounded x / scale of every K value written (NaN elsewhere)."""
    bs = k_cache.shape[1]
    out = {"k": (np.array(k_cache), np.array(k_scale, dtype=np.float64)),
           "v": (np.array(v_cache), np.array(v_scale, dtype=np.float64))}
    k_exact = np.full(k_cache.shape, np.nan)
    q_rot = np.array(q)
    for b in range(len(context_lens)):
        t0, t1 = int(query_start_loc[b]), int(query_start_loc[b + 1])
        ctx = int(context_lens[b])
        first = ctx - (t1 - t0)
        if t1 == t0:
            continue
        pos = np.arange(first, ctx)
        q_rot[t0:t1] = f64_to_bf16_bits(rope64(bf16_bits_to_f64(q[t0:t1]), pos[:, None], rope_theta))
        x = {"k": rope64(bf16_bits_to_f64(k[t0:t1]), pos[:, None], rope_theta), "v": bf16_bits_to_f64(v[t0:t1])}
        for j in range(first // bs, (ctx - 1) // bs + 1):
            blk = int(block_tables[b][j])
            lo, hi = max(first, j * bs), min(ctx, (j + 1) * bs)
            r0, r1 = lo - j * bs, hi - j * bs
            for name, (cache, scale) in out.items():
                fresh = x[name][lo - first:hi - first]
                mag = np.where(np.isfinite(fresh), np.abs(fresh), 0.0)
                s = scale_for(mag.max(axis=(0, 2)), kind)
                if r0 > 0:
                    s = np.maximum(s, scale[blk])
                    ratio = np.where(scale[blk] < s, scale[blk] / s, 1.0)
                    cache[blk, :r0] = encode(decode(cache[blk, :r0], kind) * ratio[:, None], kind)
                cache[blk, r0:r1] = encode(fresh / s[:, None], kind)
                if name == "k":
                    k_exact[blk, r0:r1] = fresh / s[:, None]
                scale[blk] = s
    return q_rot, out["k"][0], out["v"][0], out["k"][1], out["v"][1], k_exact
