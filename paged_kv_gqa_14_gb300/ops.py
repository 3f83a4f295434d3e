"""Python binding with the C-ABI's names: argument marshalling only.

Every function here checks dtypes/devices, turns torch tensors into pointers, sizes and
element strides, and calls the matching ``pkv_*`` entry point on the current torch CUDA
stream.  No arithmetic of the path runs in Python or torch: all of it is in the kernels.
PyTorch supplies device memory (the output and workspace buffers) and the stream.
"""

from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _lib

BLOCK_SIZE = 16  # the pool's default block size
SUPPORTED_BLOCK_SIZES = (8, 16, 32, 64, 128)


# The current stream's raw handle without building a torch.cuda.Stream object (about 0.1 us
# instead of 3 us per call on the Grace host); torch.cuda.current_stream() where torch lacks it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_cur_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream_ptr(stream):
    if stream is None and _raw_stream is not None and _cur_device is not None:
        return ctypes.c_void_p(_raw_stream(_cur_device()))
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _allocating_on(stream):
    """Tensors made inside belong to ``stream``: torch reuses a freed one for that stream's later work only, and so
    not while the call that it was made for still runs there."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _new_output(like, shape, stream):
    """A bf16 output for a call on ``stream``: its memory comes from that stream's, where nothing else still uses it,
    and goes back only when the current stream, whose caller gets it, is done with it too."""
    if stream is None:
        return like.new_empty(shape)
    with _allocating_on(stream):
        out = like.new_empty(shape)
    if out.is_cuda:  # (else refused further on)
        out.record_stream(torch.cuda.current_stream())
    return out


def _need(t, name, dtype, ndim):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")


def _rows(t, name):
    """(token stride, head stride) of a [T, H, d] tensor whose last dim is contiguous."""
    if t.stride(2) != 1:
        raise ValueError(f"{name}: head_dim must be contiguous")
    return t.stride(0), t.stride(1)


def _contig1(t, name):
    if t.dim() != 1 or (t.numel() > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous 1-D tensor")


def kv_append(q, k, v, positions, slot_mapping, k_cache, v_cache, rope_theta, stream=None):
    """Fused RoPE + KV append (``pkv_kv_append``).  q is rotated in place."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k, "k", torch.bfloat16, 3)
    _need(v, "v", torch.bfloat16, 3)
    _need(positions, "positions", torch.int64, 1)
    _need(slot_mapping, "slot_mapping", torch.int64, 1)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _contig1(positions, "positions")
    _contig1(slot_mapping, "slot_mapping")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("k_cache / v_cache must be contiguous [num_blocks, block_size, Hkv, d]")
    if k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache differ in shape")
    T, hq, d = q.shape
    nb, bs, hkv, dc = k_cache.shape
    if k.shape != (T, hkv, d) or v.shape != (T, hkv, d) or dc != d:
        raise ValueError("k / v / cache shapes disagree with q")
    if positions.shape[0] != T or slot_mapping.shape[0] != T:
        raise ValueError("positions / slot_mapping must have num_tokens entries")
    qs, qh = _rows(q, "q")
    ks, kh = _rows(k, "k")
    vs, vh = _rows(v, "v")
    st = _lib.load().pkv_kv_append(
        q.data_ptr(), qs, qh, k.data_ptr(), ks, kh, v.data_ptr(), vs, vh,
        positions.data_ptr(), slot_mapping.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        T, hq, hkv, d, nb, bs, float(rope_theta), _stream_ptr(stream))
    _lib.check("pkv_kv_append", st)


def kv_append_paged(q, k, v, block_tables, context_lens, query_start_loc, k_cache, v_cache, rope_theta,
                    positions_out=None, slot_mapping_out=None, max_blocks_per_seq=None, stream=None):
    """kv_append with positions and slots derived on the GPU from the scheduler's tables
    (``pkv_kv_append_paged``).  q is rotated in place."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k, "k", torch.bfloat16, 3)
    _need(v, "v", torch.bfloat16, 3)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    _need(query_start_loc, "query_start_loc", torch.int32, 1)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _contig1(context_lens, "context_lens")
    _contig1(query_start_loc, "query_start_loc")
    if block_tables.stride(1) != 1:
        raise ValueError("block_tables rows must be contiguous")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("k_cache / v_cache must be contiguous [num_blocks, block_size, Hkv, d]")
    T, hq, d = q.shape
    nb, bs, hkv, dc = k_cache.shape
    if k.shape != (T, hkv, d) or v.shape != (T, hkv, d) or dc != d or v_cache.shape != k_cache.shape:
        raise ValueError("k / v / cache shapes disagree with q")
    B = context_lens.shape[0]
    if query_start_loc.shape[0] != B + 1 or block_tables.shape[0] != B:
        raise ValueError("query_start_loc must have num_seqs + 1 entries, block_tables num_seqs rows")
    for name, t in (("positions_out", positions_out), ("slot_mapping_out", slot_mapping_out)):
        if t is not None:
            _need(t, name, torch.int64, 1)
            _contig1(t, name)
            if t.shape[0] != T:
                raise ValueError(f"{name} must have num_tokens entries")
    mb = block_tables.shape[1] if max_blocks_per_seq is None else int(max_blocks_per_seq)
    qs, qh = _rows(q, "q")
    ks, kh = _rows(k, "k")
    vs, vh = _rows(v, "v")
    st = _lib.load().pkv_kv_append_paged(
        q.data_ptr(), qs, qh, k.data_ptr(), ks, kh, v.data_ptr(), vs, vh, block_tables.data_ptr(),
        block_tables.stride(0), mb, context_lens.data_ptr(), query_start_loc.data_ptr(), B, k_cache.data_ptr(),
        v_cache.data_ptr(), T, hq, hkv, d, nb, bs, float(rope_theta),
        None if positions_out is None else positions_out.data_ptr(),
        None if slot_mapping_out is None else slot_mapping_out.data_ptr(), _stream_ptr(stream))
    _lib.check("pkv_kv_append_paged", st)


def rope_turn_table(rope_theta, head_dim):
    """The rotation frequencies kv_append uses, as uint64 0.64 fixed-point turn fractions
    (``pkv_rope_turn_table``; host only, no GPU)."""
    import numpy as np

    out = (ctypes.c_uint64 * (int(head_dim) // 2 or 1))()
    _lib.check("pkv_rope_turn_table", _lib.load().pkv_rope_turn_table(float(rope_theta), int(head_dim), out))
    return np.frombuffer(out, dtype=np.uint64)[: int(head_dim) // 2].copy()


def workspace_size(num_tokens, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, decode_ctas=0,
                   diff=False):
    """Bytes of workspace ``paged_attention`` needs (``pkv_paged_attention_workspace_size_ex``;
    ``decode_ctas`` as the per-call option, 0 for the process default), or with ``diff`` those of
    ``paged_attention_diff`` (``pkv_paged_attention_diff_workspace_size``)."""
    size = (_lib.load().pkv_paged_attention_diff_workspace_size if diff
            else _lib.load().pkv_paged_attention_workspace_size_ex)
    n = size(num_tokens, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, int(decode_ctas))
    if n == 0:
        raise ValueError("invalid sizes for paged_attention")
    return int(n)


def alloc_workspace(num_tokens, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                    device=None, decode_ctas=0, diff=False):
    """A caller-owned workspace tensor (uint8) of the required size on `device` (default: the
    current CUDA device); torch's caching allocator returns 512-byte aligned blocks.  ``diff``: for
    ``paged_attention_diff`` (it serves the other attentions of these sizes as well)."""
    n = workspace_size(num_tokens, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, decode_ctas,
                       diff)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


_OVERLAP = {None: 0, True: 1, False: 2}
PLAN_EARLY = 1  # PKV_ATTN_PLAN_EARLY
STREAM_EARLY = 2  # PKV_ATTN_STREAM_EARLY


STREAM_EARLY_MIN_KEYS = 1 << 17


def stream_early_pays(num_seqs, max_blocks_per_seq, block_size):
    """Whether PKV_ATTN_STREAM_EARLY is worth setting for a batch of this size: the decode then
    reads the plan through a published word, one round trip to L2 later than through the
    planner's end, which costs about 1 us on a batch that is latency-bound anyway and is repaid
    once the pages a decode CTA can copy during the append dominate (append + attention step on
    one GB300: 32 sequences of up to 1152 keys, L2 flushed, 20.1 -> 21.2 us; 256 of up to 2048,
    156.2 -> 154.0 us; 50 of 8192, 133.9 -> 132.5 us).  The rule: at least STREAM_EARLY_MIN_KEYS
    key slots in the block tables."""
    return num_seqs * max_blocks_per_seq * block_size >= STREAM_EARLY_MIN_KEYS


def attention_options(options):
    """A pkv_attention_options from a dict (build it once and pass it to every call):
    decode_kernel ('auto' | 'simt' | 'tensor'), prefill_kernel ('auto' | 'mma' | 'tcgen05'),
    overlap (None | True | False), decode_ctas (int), plan_early (bool: PKV_ATTN_PLAN_EARLY),
    stream_early (bool: PKV_ATTN_STREAM_EARLY; both flags are defined in include/pkv.h),
    side_stream (torch.cuda.Stream) with fork_event and join_event (torch.cuda.Event)."""
    if options is None or isinstance(options, _lib.AttentionOptions):
        return options  # (a struct built earlier is passed through: no per-call marshalling)
    unknown = set(options) - {"decode_kernel", "prefill_kernel", "overlap", "decode_ctas", "plan_early",
                              "stream_early", "side_stream", "fork_event", "join_event"}
    if unknown:
        raise ValueError(f"unknown options {sorted(unknown)}")
    opt = _lib.AttentionOptions()
    opt.struct_size = ctypes.sizeof(_lib.AttentionOptions)
    opt.decode_kernel = DECODE_KERNELS[options.get("decode_kernel", "auto")]
    opt.prefill_kernel = PREFILL_KERNELS[options.get("prefill_kernel", "auto")]
    opt.overlap = _OVERLAP[options.get("overlap", None)]
    opt.decode_ctas = int(options.get("decode_ctas", 0))
    opt.flags = (PLAN_EARLY if options.get("plan_early", False) else 0) | (
        STREAM_EARLY if options.get("stream_early", False) else 0)
    side = options.get("side_stream")
    if side is not None:
        fork, join = options.get("fork_event"), options.get("join_event")
        for ev in (fork, join):  # torch creates an event's CUDA handle at its first record
            if ev is not None and not ev.cuda_event:
                ev.record(side)
        opt.side_stream = ctypes.c_void_p(side.cuda_stream)
        opt.fork_event = ctypes.c_void_p(fork.cuda_event) if fork is not None else None
        opt.join_event = ctypes.c_void_p(join.cuda_event) if join is not None else None
    return opt


def paged_attention(q, k_cache, v_cache, block_tables, context_lens, query_start_loc, scale, out=None,
                    workspace=None, max_blocks_per_seq=None, stream=None, options=None):
    """Paged GQA over a ragged prefill/decode batch (``pkv_paged_attention``, or with per-call
    ``options`` -- a dict or a struct from ``attention_options`` -- ``pkv_paged_attention_ex``).
    A workspace that is not given belongs to the call's stream, an output to it and the current one.  Returns out."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    _need(query_start_loc, "query_start_loc", torch.int32, 1)
    _contig1(context_lens, "context_lens")
    _contig1(query_start_loc, "query_start_loc")
    if block_tables.stride(1) != 1:
        raise ValueError("block_tables rows must be contiguous")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("k_cache / v_cache must be contiguous [num_blocks, block_size, Hkv, d]")
    T, hq, d = q.shape
    nb, bs, hkv, dc = k_cache.shape
    if dc != d or v_cache.shape != k_cache.shape:
        raise ValueError("cache shapes disagree with q")
    B = context_lens.shape[0]
    if query_start_loc.shape[0] != B + 1 or block_tables.shape[0] != B:
        raise ValueError("query_start_loc must have num_seqs + 1 entries, block_tables num_seqs rows")
    mb = block_tables.shape[1] if max_blocks_per_seq is None else int(max_blocks_per_seq)
    if out is None:
        out = _new_output(q, q.shape, stream)
    _need(out, "out", torch.bfloat16, 3)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    opt = attention_options(options)
    if workspace is None:
        with _allocating_on(stream):
            workspace = alloc_workspace(T, B, hq, hkv, d, mb, device=q.device,
                                        decode_ctas=opt.decode_ctas if opt is not None else 0)
    qs, qh = _rows(q, "q")
    os_, oh = _rows(out, "out")
    args = (q.data_ptr(), qs, qh, k_cache.data_ptr(), v_cache.data_ptr(), nb, bs,
            block_tables.data_ptr(), block_tables.stride(0), mb, context_lens.data_ptr(),
            query_start_loc.data_ptr(), B, out.data_ptr(), os_, oh, T, hq, hkv, d, float(scale),
            workspace.data_ptr(), workspace.numel(), _stream_ptr(stream))
    if opt is None:
        _lib.check("pkv_paged_attention", _lib.load().pkv_paged_attention(*args))
    else:
        _lib.check("pkv_paged_attention_ex", _lib.load().pkv_paged_attention_ex(*args, ctypes.byref(opt)))
    return out


# ------------------------------------------------------------------ the 8-bit cache
Q8_FORMATS = {torch.int8: 1, torch.float8_e4m3fn: 2}  # PKV_Q8_INT8, PKV_Q8_E4M3


def alloc_q8_cache(num_blocks, block_size, num_kv_heads, head_dim, dtype=torch.int8, device=None):
    """The tensors of an 8-bit cache: k_cache, v_cache [num_blocks, block_size, Hkv, d] of ``dtype``
    (torch.int8 or torch.float8_e4m3fn) and k_scale, v_scale float32 [num_blocks, Hkv].  Nothing is
    initialised: kv_append_q8 writes a block's rows and scale before anything reads them."""
    if dtype not in Q8_FORMATS:
        raise TypeError(f"dtype must be one of {list(Q8_FORMATS)}, got {dtype}")
    device = device or "cuda"
    pools = [torch.empty(num_blocks, block_size, num_kv_heads, head_dim, dtype=dtype, device=device) for _ in "kv"]
    scales = [torch.empty(num_blocks, num_kv_heads, dtype=torch.float32, device=device) for _ in "kv"]
    return (*pools, *scales)


# The calls below go through a small extension in C (csrc/q8_call.c), which checks the tensors and calls the
# library; where a check fails, the same checks follow here one by one to say what is wrong.
_BF16, _I32, _F32 = torch.bfloat16, torch.int32, torch.float32


def _refuse_numbers(max_blocks_per_seq, **numbers):
    for name, x in numbers.items():
        if isinstance(x, (str, bytes)) or not (hasattr(x, "__float__") or hasattr(x, "__index__")):
            raise TypeError(f"{name} must be a number, got {type(x).__name__}")
    if max_blocks_per_seq is not None and not hasattr(max_blocks_per_seq, "__index__"):
        raise TypeError(f"max_blocks_per_seq must be an integer, got {type(max_blocks_per_seq).__name__}")


def _refuse_tables(block_tables, context_lens, start_loc, start_name, max_blocks_per_seq):
    _need(block_tables, "block_tables", _I32, 2)
    _need(context_lens, "context_lens", _I32, 1)
    _need(start_loc, start_name, _I32, 1)
    _contig1(context_lens, "context_lens")
    _contig1(start_loc, start_name)
    if block_tables.stride(1) != 1 and block_tables.shape[1] > 1:
        raise ValueError("block_tables rows must be contiguous")
    B = context_lens.shape[0]
    if start_loc.shape[0] != B + 1 or block_tables.shape[0] != B:
        raise ValueError(f"{start_name} must have num_seqs + 1 entries, block_tables num_seqs rows")
    if max_blocks_per_seq is not None and int(max_blocks_per_seq) > block_tables.shape[1]:
        raise ValueError("max_blocks_per_seq is more than block_tables' columns")


def _refuse_rest(named):
    """Raises for the device of the first tensor that is elsewhere, or else for the shapes."""
    cur = torch.cuda.current_device()
    for name, t in named.items():
        if t.device.index != cur:
            raise ValueError(f"{name} is on {t.device}, the current device is cuda:{cur}")
    raise ValueError("shapes disagree: " + ", ".join(f"{n} {tuple(t.shape)}" for n, t in named.items()))


def _refuse_q8(rows, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, start_loc, start_name,
               max_blocks_per_seq, **numbers):
    """Raises for the first thing wrong with a call on an 8-bit cache; ``rows``: its [rows, heads, d] bf16
    tensors by name."""
    _refuse_numbers(max_blocks_per_seq, **numbers)
    if not isinstance(k_cache, torch.Tensor):
        raise TypeError("k_cache must be a torch.Tensor")
    if k_cache.dtype not in Q8_FORMATS:
        raise TypeError(f"k_cache must be one of {list(Q8_FORMATS)}, got {k_cache.dtype}")
    _need(k_cache, "k_cache", k_cache.dtype, 4)
    _need(v_cache, "v_cache", k_cache.dtype, 4)
    _need(k_scale, "k_scale", _F32, 2)
    _need(v_scale, "v_scale", _F32, 2)
    for name, t in rows.items():
        _need(t, name, _BF16, 3)
        _rows(t, name)
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("k_cache / v_cache must be contiguous [num_blocks, block_size, Hkv, d]")
    if not (k_scale.is_contiguous() and v_scale.is_contiguous()):
        raise ValueError("k_scale / v_scale must be contiguous [num_blocks, Hkv]")
    nb, _, hkv, _ = k_cache.shape
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache differ in shape")
    if k_scale.shape != (nb, hkv) or v_scale.shape != (nb, hkv):
        raise ValueError("k_scale / v_scale must be [num_blocks, Hkv]")
    _refuse_tables(block_tables, context_lens, start_loc, start_name, max_blocks_per_seq)
    _refuse_rest({**rows, "k_cache": k_cache, "v_cache": v_cache, "k_scale": k_scale, "v_scale": v_scale,
                  "block_tables": block_tables, "context_lens": context_lens, start_name: start_loc})


def _where(stream):
    """(raw handle of the stream, current device); device -2, no tensor's, where there is no GPU."""
    try:
        dev = _cur_device() if _cur_device is not None else torch.cuda.current_device()
        if stream is not None:
            return stream.cuda_stream, dev
        return (_raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream), dev
    except RuntimeError:
        return 0, -2


def kv_append_q8(q, k, v, block_tables, context_lens, query_start_loc, k_cache, v_cache, k_scale, v_scale, rope_theta,
                 max_blocks_per_seq=None, stream=None):
    """Fused RoPE, quantisation and append into an 8-bit cache (``pkv_kv_append_q8``), each token's
    place derived on the GPU from the scheduler's tables.  q is rotated in place; the caches are int8 or
    float8_e4m3fn with one power-of-two scale per block and kv head."""
    st = _lib.q8call().append(q, k, v, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                              query_start_loc, rope_theta, max_blocks_per_seq, *_where(stream))
    if st < 0:
        _refuse_q8({"q": q, "k": k, "v": v}, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                   query_start_loc, "query_start_loc", max_blocks_per_seq, rope_theta=rope_theta)
    if st:
        _lib.check("pkv_kv_append_q8", st)


def kv_read_q8(k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, read_start_loc, k_out, v_out,
               max_blocks_per_seq=None, stream=None):
    """The last ``read_start_loc[b+1] - read_start_loc[b]`` tokens of every sequence of an 8-bit cache
    as bf16 (``pkv_kv_read_q8``), into rows ``read_start_loc[b]`` on of k_out and v_out [rows, Hkv, d].
    Returns (k_out, v_out)."""
    st = _lib.q8call().read(k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, read_start_loc,
                            k_out, v_out, max_blocks_per_seq, *_where(stream))
    if st < 0:
        _refuse_q8({"k_out": k_out, "v_out": v_out}, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                   read_start_loc, "read_start_loc", max_blocks_per_seq)
    if st:
        _lib.check("pkv_kv_read_q8", st)
    return k_out, v_out


def paged_attention_q8(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, query_start_loc, scale,
                       out=None, workspace=None, max_blocks_per_seq=None, stream=None, options=None):
    """Paged GQA over an 8-bit cache (``pkv_paged_attention_q8``): as ``paged_attention``, K and V being
    what the cache stands for.  ``options`` as there; the "simt" decode and the "mma" prefill are refused.
    ``workspace``: a uint8 tensor from ``alloc_workspace``.  Returns out."""
    opt = None if options is None else attention_options(options)
    if out is None or workspace is None:
        rows = {"q": q} if out is None else {"q": q, "out": out}
        if not (isinstance(q, torch.Tensor) and q.dim() == 3 and isinstance(k_cache, torch.Tensor) and k_cache.dim() == 4
                and isinstance(block_tables, torch.Tensor) and block_tables.dim() == 2
                and isinstance(context_lens, torch.Tensor) and context_lens.dim() == 1):
            _refuse_q8(rows, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, query_start_loc,
                       "query_start_loc", max_blocks_per_seq, scale=scale)
        if out is None:
            out = _new_output(q, q.shape, stream)
        if workspace is None:
            T, hq, d = q.shape
            with _allocating_on(stream):
                workspace = alloc_workspace(T, context_lens.shape[0], hq, k_cache.shape[2], d, block_tables.shape[1],
                                            device=q.device, decode_ctas=opt.decode_ctas if opt is not None else 0)
    st = _lib.q8call().attention(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, query_start_loc,
                                 out, workspace, scale, max_blocks_per_seq,
                                 0 if opt is None else ctypes.addressof(opt), *_where(stream))
    if st < 0:
        if isinstance(k_cache, torch.Tensor) and not (
                isinstance(workspace, torch.Tensor) and workspace.dim() == 1 and workspace.is_contiguous()
                and workspace.device == k_cache.device):
            raise ValueError("workspace must be a contiguous 1-D uint8 tensor on the cache's device")
        _refuse_q8({"q": q, "out": out}, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                   query_start_loc, "query_start_loc", max_blocks_per_seq, scale=scale)
    if st:
        _lib.check("pkv_paged_attention_q8", st)
    return out


# ------------------------------------------------------------------ attention variants
def _whole(x, name):
    n = int(x)
    if n != x:
        raise ValueError(f"{name} must hold whole numbers, got {x!r}")
    return n


def relative_buckets(num_buckets=None, max_distance=None, starts=None):
    """The buckets of ``paged_attention_bias`` (a pkv_relative_buckets; build it once and pass it to every call):
    either the usual ones of ``num_buckets`` and ``max_distance`` (``pkv_relative_buckets_log``), or the
    least distance of each bucket in ``starts``, a sequence that begins with 0 and does not fall."""
    b = _lib.RelativeBuckets()
    if starts is None:
        if num_buckets is None or max_distance is None:
            raise ValueError("relative_buckets needs num_buckets and max_distance, or starts")
        sizes = _whole(num_buckets, "num_buckets"), _whole(max_distance, "max_distance")
        if not all(-(2**31) <= x < 2**31 for x in sizes):
            raise ValueError(f"num_buckets and max_distance must fit 32 bits, got {sizes}")
        st = _lib.load().pkv_relative_buckets_log(*sizes, ctypes.byref(b))
        _lib.check("pkv_relative_buckets_log", st)
        return b
    if num_buckets is not None or max_distance is not None:
        raise ValueError("relative_buckets takes num_buckets and max_distance, or starts, not both")
    starts = [_whole(x, "starts") for x in starts]
    if not 1 <= len(starts) <= _lib.MAX_BUCKETS:
        raise ValueError(f"starts must have 1 to {_lib.MAX_BUCKETS} entries, got {len(starts)}")
    if starts[0] != 0 or any(y < x for x, y in zip(starts, starts[1:])) or starts[-1] > 2**31 - 1:
        raise ValueError("starts must begin with 0, not fall and fit 32 bits")
    b.struct_size = ctypes.sizeof(b)
    b.num_buckets = len(starts)
    b.starts[: len(starts)] = starts
    return b


def _refuse_variant(q, k_cache, v_cache, block_tables, context_lens, query_start_loc, out, workspace,
                    max_blocks_per_seq, more, diff=False, **numbers):
    """Raises for the first thing wrong with a call of an attention variant; ``more``: its own tensors."""
    _refuse_numbers(max_blocks_per_seq, **numbers)
    _need(q, "q", _BF16, 3)
    _rows(q, "q")
    _need(k_cache, "k_cache", _BF16, 4)
    _need(v_cache, "v_cache", _BF16, 4)
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("k_cache / v_cache must be contiguous [num_blocks, block_size, Hkv, d]")
    if v_cache.shape != k_cache.shape or k_cache.shape[3] != q.shape[2]:
        raise ValueError("cache shapes disagree with q")
    _refuse_tables(block_tables, context_lens, query_start_loc, "query_start_loc", max_blocks_per_seq)
    T, hq, d = q.shape
    if diff and hq % 2:
        raise ValueError("q must have an even number of heads")
    _need(out, "out", _BF16, 3)
    _rows(out, "out")
    want = (T, hq // 2, 2 * d) if diff else (T, hq, d)
    if out.shape != want:
        raise ValueError(f"out must be {want}, got {tuple(out.shape)}")
    if not (isinstance(workspace, torch.Tensor) and workspace.dim() == 1 and workspace.is_contiguous()
            and workspace.device == k_cache.device):
        raise ValueError("workspace must be a contiguous 1-D uint8 tensor on the cache's device")
    for name, (t, dtypes, shapes) in more.items():
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype not in dtypes:
            raise TypeError(f"{name} must be one of {list(dtypes)}, got {t.dtype}")
        if tuple(t.shape) not in shapes:
            raise ValueError(f"{name} must be {' or '.join(str(x) for x in shapes)}, got {tuple(t.shape)}")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError(f"{name}: the last dim must be contiguous")
    _refuse_rest({"q": q, "k_cache": k_cache, "v_cache": v_cache, "block_tables": block_tables,
                  "context_lens": context_lens, "query_start_loc": query_start_loc, "out": out,
                  **{n: t for n, (t, _, _) in more.items()}})


def _variant_buffers(q, k_cache, block_tables, context_lens, out, workspace, opt, stream, diff):
    """The output and workspace of a call that were not given; None where the tensors they follow are wrong."""
    if not (isinstance(q, torch.Tensor) and q.dim() == 3 and q.is_cuda and isinstance(k_cache, torch.Tensor)
            and k_cache.dim() == 4 and isinstance(block_tables, torch.Tensor) and block_tables.dim() == 2
            and isinstance(context_lens, torch.Tensor) and context_lens.dim() == 1):
        return out, workspace
    T, hq, d = q.shape
    hkv = k_cache.shape[2]
    if out is None:
        out = _new_output(q, (T, hq // 2, 2 * d) if diff else (T, hq, d), stream)
    if workspace is None and hq > 0 and hkv > 0 and not (diff and (hq % 2 or hkv % 2)):
        with _allocating_on(stream):
            workspace = alloc_workspace(T, context_lens.shape[0], hq, hkv, d, block_tables.shape[1], device=q.device,
                                        decode_ctas=opt.decode_ctas if opt is not None else 0, diff=diff)
    return out, workspace


def paged_attention_bias(q, k_cache, v_cache, block_tables, context_lens, query_start_loc, scale, bias, buckets,
                         out=None, workspace=None, max_blocks_per_seq=None, stream=None, options=None):
    """Paged GQA with a learned relative position bias by buckets (``pkv_paged_attention_bias``): as
    ``paged_attention``, with ``bias[bucket(n), h]`` added to the score of q head h and the key at distance n.
    ``bias``: [num_buckets, Hq], float32 or bfloat16; ``buckets`` from ``relative_buckets``.  A bias of -inf takes
    the key out; a row without keys left gives zeros.  ``options`` as for ``paged_attention``; the "simt"
    decode and the "mma" prefill are refused.  What is not given belongs to the streams as there.  Returns out."""
    opt = None if options is None else attention_options(options)
    if not isinstance(buckets, _lib.RelativeBuckets):
        raise TypeError(f"buckets must come from relative_buckets, got {type(buckets).__name__}")
    if out is None or workspace is None:
        out, workspace = _variant_buffers(q, k_cache, block_tables, context_lens, out, workspace, opt, stream, False)
    st = _lib.q8call().bias(q, k_cache, v_cache, block_tables, context_lens, query_start_loc, out, workspace, scale,
                            bias, ctypes.addressof(buckets), max_blocks_per_seq,
                            0 if opt is None else ctypes.addressof(opt), *_where(stream))
    if st < 0:
        shape = (buckets.num_buckets, q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else -1)
        _refuse_variant(q, k_cache, v_cache, block_tables, context_lens, query_start_loc, out, workspace,
                        max_blocks_per_seq, {"bias": (bias, (_F32, _BF16), (shape,))}, scale=scale)
    if st:
        _lib.check("pkv_paged_attention_bias", st)
    return out


def paged_attention_diff(q, k_cache, v_cache, block_tables, context_lens, query_start_loc, scale, lam,
                         norm_weight=None, norm_eps=1e-5, out_scale=1.0, out=None, workspace=None,
                         max_blocks_per_seq=None, stream=None, options=None):
    """Differential attention over the paged cache (``pkv_paged_attention_diff``): head h of Hq / 2 weighs the values
    of its kv pair (v heads 2g and 2g + 1 side by side, g = h // (Hq // Hkv)) with the softmax map of q head 2h and
    k head 2g less ``lam[h]`` times that of q head 2h + 1 and k head 2g + 1, over spans as in ``paged_attention``.
    ``lam``: float32, [Hq / 2] or [T, Hq / 2].  With ``norm_weight`` (float32 [2 d]) each head's 2 d numbers are
    RMS-normalised and multiplied by it, and by ``out_scale`` in any case.  ``workspace``: from
    ``alloc_workspace(..., diff=True)``.  ``options`` as for ``paged_attention_bias``.  What is not given belongs to the
    streams as for ``paged_attention``.  Returns out [T, Hq / 2, 2 d]."""
    opt = None if options is None else attention_options(options)
    if out is None or workspace is None:
        out, workspace = _variant_buffers(q, k_cache, block_tables, context_lens, out, workspace, opt, stream, True)
    st = _lib.q8call().diff(q, k_cache, v_cache, block_tables, context_lens, query_start_loc, out, workspace, scale,
                            lam, norm_weight, norm_eps, out_scale, max_blocks_per_seq,
                            0 if opt is None else ctypes.addressof(opt), *_where(stream))
    if st < 0:
        T, hq, d = q.shape if isinstance(q, torch.Tensor) and q.dim() == 3 else (-1, -2, -1)
        more = {"lam": (lam, (_F32,), ((hq // 2,), (T, hq // 2)))}
        if norm_weight is not None:
            more["norm_weight"] = (norm_weight, (_F32,), ((2 * d,),))
        _refuse_variant(q, k_cache, v_cache, block_tables, context_lens, query_start_loc, out, workspace,
                        max_blocks_per_seq, more, diff=True, scale=scale, norm_eps=norm_eps, out_scale=out_scale)
    if st:
        _lib.check("pkv_paged_attention_diff", st)
    return out


def set_decode_ctas(n):
    """Override the decode split-K grid (0 = one CTA per SM).  Process-wide."""
    _lib.check("pkv_set_decode_ctas", _lib.load().pkv_set_decode_ctas(int(n)))


def set_overlap(on):
    """Run a mixed batch's prefill tiles beside the decode on a second stream (True, the
    default) or before it on the caller's stream (False).  Process-wide."""
    _lib.check("pkv_set_overlap", _lib.load().pkv_set_overlap(1 if on else 0))


DECODE_KERNELS = {"auto": 0, "simt": 1, "tensor": 2}


def set_decode_kernel(kind):
    """Decode arithmetic for later calls: "auto", "simt" (CUDA cores) or "tensor" (mma.sync)."""
    _lib.check("pkv_set_decode_kernel", _lib.load().pkv_set_decode_kernel(DECODE_KERNELS[kind]))


PREFILL_KERNELS = {"auto": 0, "mma": 1, "tcgen05": 2}


def set_prefill_kernel(kind):
    """Prefill-tile arithmetic for later calls: "auto", "mma" (mma.sync) or "tcgen05"."""
    _lib.check("pkv_set_prefill_kernel", _lib.load().pkv_set_prefill_kernel(PREFILL_KERNELS[kind]))


def set_fault_injection(kind):
    """Test only (``pkv_set_fault_injection``): ``"decode_no_copies"`` makes the decode producer
    issue nothing, so its consumers' bounded waits run out; ``"plan_no_ready"`` keeps the
    planner from publishing its ready word under ``stream_early``, so the decode's bounded polls
    run out and it falls back to the planner's end; ``"prefill_no_copies"`` is the first for the prefill tiles over
    an 8-bit cache and of the attention variants; ``None`` turns it off."""
    code = {None: 0, "decode_no_copies": 1, "plan_no_ready": 2, "prefill_no_copies": 4}[kind]
    _lib.check("pkv_set_fault_injection", _lib.load().pkv_set_fault_injection(code))


def get_device_error(clear=True, stream=None):
    """Synchronise the stream and return the or-ed PKV_DEVERR_* bits of the current device."""
    bits = ctypes.c_uint32(0)
    st = _lib.load().pkv_get_device_error(ctypes.byref(bits), 1 if clear else 0, _stream_ptr(stream))
    _lib.check("pkv_get_device_error", st)
    return int(bits.value)


def set_kernel_events(kernel, start=None, stop=None):
    """Record torch.cuda.Event ``start``/``stop`` around every launch of ``kernel``
    ("kv_append", "plan", "prefill", "decode"); None switches it off."""
    which = _lib.KERNELS[kernel]
    for e in (start, stop):
        if e is not None and e.cuda_event == 0:
            e.record()  # torch creates the CUDA event lazily, on its first record
    sp = ctypes.c_void_p(start.cuda_event) if start is not None else None
    ep = ctypes.c_void_p(stop.cuda_event) if stop is not None else None
    _lib.check("pkv_set_kernel_events", _lib.load().pkv_set_kernel_events(which, sp, ep))


def copy(dst, src, stream=None):
    """Byte copy src -> dst by a kernel (``pkv_copy``); either tensor may be on the device or in
    pinned host memory.  Both must be contiguous, of equal byte size, 16-byte aligned."""
    for name, t in (("dst", dst), ("src", src)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if not t.is_cuda and not t.is_pinned():
            raise ValueError(f"{name} must be a CUDA tensor or pinned host memory")
    nbytes = dst.numel() * dst.element_size()
    if src.numel() * src.element_size() != nbytes:
        raise ValueError("dst and src differ in byte size")
    _lib.check("pkv_copy", _lib.load().pkv_copy(dst.data_ptr(), src.data_ptr(), nbytes, _stream_ptr(stream)))
    return dst

