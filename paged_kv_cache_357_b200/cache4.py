"""The 4-bit cache and its eviction: torch-facing wrappers of libpa's
pa_*_fp4, pa_decode_weights and pa_evict (C ABI in include/pa.h).

Argument marshalling only, as in ``_lib``: tensors are checked for device,
dtype, shape and contiguity, and non-zero return codes become ``PaError``.
The calls run on the tensors' device, whichever is current, and on its
current stream unless one is given.

A 4-bit pool is uint8 ``[num_blocks, num_kv_heads, block_size, head_dim * 9 // 16]``
(``fp4_pool_shape``).  The last two dimensions together are one tile of bytes
(all the rows' codes, then all the rows' scales), not rows of their own.
"""

from __future__ import annotations

import ctypes
from functools import lru_cache
from typing import Tuple

from ._lib import (PA_BF16, PA_EVICT_TEST_WITHHOLD, PA_FP16, DecodeOpts, PaError, PoolDesc, TokenWeights, _dtype_code,
                   _need, _ptr, _torch, load, pool_desc)

# bound at the first call, with torch and the library loaded (_bind)
torch = None
_codes = {}             # 16-bit dtype -> its code in a descriptor
_raw_stream = None      # device index -> handle of its current stream
_current_device = None  # -> index of the current device
_lib = None


def _bind() -> None:
    global torch, _raw_stream, _current_device, _lib
    t = _torch()
    _lib = load()
    _codes.update({t.float16: PA_FP16, t.bfloat16: PA_BF16})
    # the handle without a Stream object around it, where this torch has it
    _raw_stream = getattr(t._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: t.cuda.current_stream(index).cuda_stream)
    _current_device = getattr(t._C, "_cuda_getDevice", None) or t.cuda.current_device
    torch = t  # last: a thread that sees it finds the rest bound


def _want(t, name, dtype, ndim, index) -> None:
    """_need for the calls of a serving loop: one line when all is well."""
    if t is None or t.dtype is not dtype or t.dim() != ndim or t.get_device() != index or not t.is_contiguous():
        _need(t, name, dtype=dtype, ndim=ndim, device=torch.device("cuda", index))


def _first(t, name, ndim) -> int:
    """The device index of a call's first tensor."""
    if torch is None:
        _bind()
    if t is None or not t.is_cuda or t.dim() != ndim or not t.is_contiguous():
        _need(t, name, ndim=ndim)
    return t.get_device()


def _stream_of(index, stream):
    if stream is None:
        return _raw_stream(index)
    if stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
    return stream.cuda_stream


def _run(where, index, fn, *args) -> None:
    """fn(*args) with the tensors' device current; PaError for its errors."""
    if _current_device() == index:
        rc = fn(*args)
    else:
        with torch.cuda.device(index):
            rc = fn(*args)
    if rc:
        raise PaError(rc, where)


def _code(t) -> int:
    code = _codes.get(t.dtype)
    return _dtype_code(t) if code is None else code  # raises


@lru_cache(maxsize=64)
def _desc_ref(nb, hkv, bs, head_dim, code):
    return ctypes.byref(PoolDesc(nb, bs, hkv, head_dim, code))


@lru_cache(maxsize=64)
def _opts_ref(num_ctas, flags):
    return ctypes.byref(DecodeOpts(num_ctas, flags))


def fp4_pool_shape(num_blocks: int, num_kv_heads: int, block_size: int, head_dim: int) -> Tuple[int, int, int, int]:
    """Shape of a uint8 pool that holds num_blocks blocks in 4 bits."""
    if block_size not in (8, 16, 32) or head_dim not in (64, 128):
        raise ValueError("4-bit pools have blocks of 8, 16 or 32 tokens and head_dim 64 or 128")
    return num_blocks, num_kv_heads, block_size, head_dim * 9 // 16


def fp4_pool_desc(pool, dtype_code: int) -> PoolDesc:
    """Descriptor of a 4-bit pool beside activations of a 16-bit type."""
    nb, hkv, bs, row = pool.shape
    return PoolDesc(nb, bs, hkv, row * 16 // 9, dtype_code)


def _want_fp4_pools(k_pool, v_pool):
    """(device index, shape) of two 4-bit pools."""
    index = _first(k_pool, "k_pool", 4)
    if k_pool.dtype is not torch.uint8:
        _need(k_pool, "k_pool", dtype=torch.uint8)
    _want(v_pool, "v_pool", torch.uint8, 4, index)
    shape = k_pool.shape
    if v_pool.shape != shape:
        raise ValueError("k_pool and v_pool shapes differ")
    if shape[3] != 72 and shape[3] != 36:
        raise ValueError("a 4-bit pool is [num_blocks, num_kv_heads, block_size, head_dim * 9 // 16]")
    return index, shape


def _want_16bit_pools(k_pool, v_pool):
    index = _first(k_pool, "k_pool", 4)
    _want(v_pool, "v_pool", k_pool.dtype, 4, index)
    shape = k_pool.shape
    if v_pool.shape != shape:
        raise ValueError("k_pool and v_pool shapes differ")
    return index, shape


def _status_ptr(dev_status, index):
    if dev_status is None:
        return None
    if dev_status.dtype is not torch.int32 or dev_status.get_device() != index or not dev_status.is_contiguous():
        _need(dev_status, "dev_status", dtype=torch.int32, device=torch.device("cuda", index))
    if dev_status.numel() < 1:
        raise ValueError("dev_status is empty")
    return dev_status.data_ptr()


def _int32(x, name) -> int:
    """x, which a C int holds (ctypes would drop the bits above)."""
    x = int(x)
    if not -(1 << 31) <= x < 1 << 31:
        raise ValueError(f"{name} does not fit 32 bits")
    return x


def _token_weights(weights, weight_rows, num_new, num_seqs, num_kv_heads, tokens, index) -> TokenWeights:
    """The pa_token_weights of weights [rows, num_kv_heads, row_tokens]."""
    _want(weights, "weights", torch.float32, 3, index)
    rows, heads, row_tokens = weights.shape
    if heads != num_kv_heads or row_tokens < tokens:
        raise ValueError("weights must be [rows, num_kv_heads, at least max_blocks_per_seq * block_size]")
    if weight_rows is not None:
        _want(weight_rows, "weight_rows", torch.int32, 1, index)
        if weight_rows.shape[0] != num_seqs:
            raise ValueError("weight_rows must have num_seqs entries")
    elif rows < num_seqs:
        raise ValueError("weights must have a row for every sequence")
    return TokenWeights(weights.data_ptr(), row_tokens, _ptr(weight_rows), rows, _int32(num_new, "num_new"))


# ---------------------------------------------------------------------------
# storage
# ---------------------------------------------------------------------------


def _want_store(k, v, slot_mapping, k_pool, v_pool):
    """(device index, tokens, pool descriptor) of a write or a read.

    When all is well one chain of conditions says so; else the checks behind
    it say what is not.  The wrappers of a serving loop's calls do this alike.
    """
    if torch is None:
        _bind()
    try:
        nb, hkv, bs, row = pool_shape = k_pool.shape
        tokens, heads, head_dim = shape = k.shape
        index, dtype = k_pool.get_device(), k.dtype
        if (index >= 0 and dtype in _codes and v.dtype is dtype and k_pool.dtype is torch.uint8
                and v_pool.dtype is torch.uint8 and slot_mapping.dtype is torch.int64 and heads == hkv
                and head_dim * 9 == row * 16 and (row == 72 or row == 36) and v.shape == shape
                and v_pool.shape == pool_shape and slot_mapping.shape == (tokens,)
                and k.get_device() == index and v.get_device() == index and v_pool.get_device() == index
                and slot_mapping.get_device() == index and k.is_contiguous() and v.is_contiguous()
                and k_pool.is_contiguous() and v_pool.is_contiguous() and slot_mapping.is_contiguous()):
            return index, tokens, _desc_ref(nb, hkv, bs, head_dim, _codes[dtype])
    except (AttributeError, TypeError, ValueError):
        pass
    index, (nb, hkv, bs, row) = _want_fp4_pools(k_pool, v_pool)
    _want(k, "k", None if k is None else k.dtype, 3, index)
    _want(v, "v", k.dtype, 3, index)
    _want(slot_mapping, "slot_mapping", torch.int64, 1, index)
    shape = k.shape
    tokens, heads, head_dim = shape
    if v.shape != shape or slot_mapping.numel() != tokens:
        raise ValueError("k, v and slot_mapping disagree on the token count")
    if heads != hkv or head_dim * 9 != row * 16:
        raise ValueError("tokens must be [T, num_kv_heads, head_dim]")
    return index, tokens, _desc_ref(nb, hkv, bs, head_dim, _code(k))


def pa_cache_write_fp4(k, v, slot_mapping, k_pool, v_pool, k_scale: float = 1.0, v_scale: float = 1.0,
                       dev_status=None, stream=None) -> None:
    """Store new tokens' K/V ([T, Hkv, D], fp16 or bf16) into their slots of 4-bit pools (pa_cache_write_fp4)."""
    index, tokens, desc = _want_store(k, v, slot_mapping, k_pool, v_pool)
    _run("pa_cache_write_fp4", index, _lib.pa_cache_write_fp4, k.data_ptr(), v.data_ptr(), slot_mapping.data_ptr(),
         tokens, k_scale, v_scale, k_pool.data_ptr(), v_pool.data_ptr(), _status_ptr(dev_status, index), desc,
         _stream_of(index, stream))


def pa_cache_read_fp4(slot_mapping, k_pool, v_pool, k, v, k_scale: float = 1.0, v_scale: float = 1.0,
                      dev_status=None, stream=None) -> None:
    """The values that 4-bit pools hold at the slots, into k, v [T, Hkv, D] (pa_cache_read_fp4)."""
    index, tokens, desc = _want_store(k, v, slot_mapping, k_pool, v_pool)
    _run("pa_cache_read_fp4", index, _lib.pa_cache_read_fp4, slot_mapping.data_ptr(), tokens, k_pool.data_ptr(),
         v_pool.data_ptr(), k_scale, v_scale, k.data_ptr(), v.data_ptr(), _status_ptr(dev_status, index), desc,
         _stream_of(index, stream))


def pa_copy_blocks_fp4(src_dst_pairs, k_pool, v_pool, dev_status=None, stream=None) -> None:
    """Copy-on-write block copies in 4-bit pools (pa_copy_blocks_fp4)."""
    index, (nb, hkv, bs, row) = _want_fp4_pools(k_pool, v_pool)
    _want(src_dst_pairs, "src_dst_pairs", torch.int64, 2, index)
    n, two = src_dst_pairs.shape
    if two != 2:
        raise ValueError("src_dst_pairs must be [n, 2]")
    _run("pa_copy_blocks_fp4", index, _lib.pa_copy_blocks_fp4, src_dst_pairs.data_ptr(), n, k_pool.data_ptr(),
         v_pool.data_ptr(), _status_ptr(dev_status, index), _desc_ref(nb, hkv, bs, row * 16 // 9, 0),
         _stream_of(index, stream))


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------


def _alloc(n: int, dev, where: str):
    if n == 0:
        raise PaError(2, where)
    return _torch().zeros(n, dtype=_torch().uint8, device=dev)


def alloc_decode_fp4_workspace(num_seqs: int, num_q_heads: int, k_pool, weights_max_blocks_per_seq: int = 0,
                               num_ctas: int = 0):
    """Zeroed workspace of pa_decode_fp4; weights_max_blocks_per_seq: the
    block tables' width when the calls pass weights, else 0."""
    desc, opts = fp4_pool_desc(k_pool, 0), DecodeOpts(num_ctas, 0)
    with _torch().cuda.device(k_pool.device):
        n = load().pa_decode_fp4_workspace_bytes(num_seqs, num_q_heads, weights_max_blocks_per_seq,
                                                 ctypes.byref(desc), ctypes.byref(opts))
    return _alloc(int(n), k_pool.device, "pa_decode_fp4_workspace_bytes")


def alloc_decode_weights_workspace(num_seqs: int, num_q_heads: int, k_pool, max_blocks_per_seq: int,
                                   num_ctas: int = 0, flags: int = 0):
    """Zeroed workspace of pa_decode_weights with the same num_ctas and flags."""
    desc, opts = pool_desc(k_pool), DecodeOpts(num_ctas, flags)
    with _torch().cuda.device(k_pool.device):
        n = load().pa_decode_weights_workspace_bytes(num_seqs, num_q_heads, max_blocks_per_seq, ctypes.byref(desc),
                                                     ctypes.byref(opts))
    return _alloc(int(n), k_pool.device, "pa_decode_weights_workspace_bytes")


def _want_decode(q, block_tables, seq_lens, out, workspace, index):
    """(num_seqs, num_q_heads, head_dim, table width, workspace bytes) of a decode."""
    try:
        S, Hq, D = shape = q.shape
        rows, width = block_tables.shape
        dtype = q.dtype
        if (rows == S and seq_lens.shape == (S,) and out.shape == shape and out.dtype is dtype
                and block_tables.dtype is torch.int32 and seq_lens.dtype is torch.int32 and q.get_device() == index
                and out.get_device() == index and block_tables.get_device() == index
                and seq_lens.get_device() == index and workspace.get_device() == index and q.is_contiguous()
                and out.is_contiguous() and block_tables.is_contiguous() and seq_lens.is_contiguous()
                and workspace.is_contiguous()):
            return S, Hq, D, width, workspace.nbytes
    except (AttributeError, TypeError, ValueError):
        pass
    _want(q, "q", q.dtype if q is not None else None, 3, index)
    shape = q.shape
    _want(out, "out", q.dtype, 3, index)
    if out.shape != shape:
        raise ValueError("out must have q's shape")
    _want(block_tables, "block_tables", torch.int32, 2, index)
    _want(seq_lens, "seq_lens", torch.int32, 1, index)
    S, width = block_tables.shape
    if S != shape[0] or seq_lens.shape[0] != S:
        raise ValueError("block_tables / seq_lens must have num_seqs rows")
    if workspace is None or workspace.get_device() != index or not workspace.is_contiguous():
        _need(workspace, "workspace", device=torch.device("cuda", index))
    return S, shape[1], shape[2], width, workspace.numel() * workspace.element_size()


def pa_decode_fp4(q, k_pool, v_pool, block_tables, seq_lens, scale: float, out, workspace, k_scale: float = 1.0,
                  v_scale: float = 1.0, lse=None, weights=None, weight_rows=None, num_new: int = 1, dev_status=None,
                  num_ctas: int = 0, stream=None) -> None:
    """pa_decode over 4-bit pools (pa_decode_fp4).  lse [num_seqs, num_q_heads]
    float32: the rows' log normalisers.  weights [rows, num_kv_heads, tokens]
    float32: the attention weights of every cached token are added to its
    entry, and set for the newest num_new tokens; sequence s has row
    weight_rows[s] (int32), or s."""
    index, (nb, hkv, bs, row) = _want_fp4_pools(k_pool, v_pool)
    S, Hq, D, width, ws_bytes = _want_decode(q, block_tables, seq_lens, out, workspace, index)
    if D * 9 != row * 16:
        raise ValueError("head_dim of q and the pools differ")
    if lse is not None:
        _want(lse, "lse", torch.float32, 2, index)
        if tuple(lse.shape) != (S, Hq):
            raise ValueError("lse must be [num_seqs, num_q_heads]")
    tw = None
    if weights is not None:
        tw = ctypes.byref(_token_weights(weights, weight_rows, num_new, S, hkv, width * bs, index))
    _run("pa_decode_fp4", index, _lib.pa_decode_fp4, q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
         block_tables.data_ptr(), width, seq_lens.data_ptr(), S, Hq, scale, k_scale, v_scale, out.data_ptr(),
         _ptr(lse), tw, workspace.data_ptr(), ws_bytes, _status_ptr(dev_status, index),
         _desc_ref(nb, hkv, bs, D, _code(q)), _opts_ref(num_ctas, 0), _stream_of(index, stream))


def pa_decode_weights(q, k_pool, v_pool, block_tables, seq_lens, scale: float, weights, out, workspace,
                      weight_rows=None, num_new: int = 1, dev_status=None, num_ctas: int = 0, flags: int = 0,
                      stream=None) -> None:
    """pa_decode over 16-bit pools that adds each cached token's attention
    weight to weights [rows, num_kv_heads, tokens] float32
    (pa_decode_weights; weight_rows and num_new as in pa_decode_fp4)."""
    index, (nb, hkv, bs, head_dim) = _want_16bit_pools(k_pool, v_pool)
    S, Hq, D, width, ws_bytes = _want_decode(q, block_tables, seq_lens, out, workspace, index)
    if q.dtype is not k_pool.dtype:
        raise TypeError(f"q must be {k_pool.dtype}, got {q.dtype}")
    if D != head_dim:
        raise ValueError("head_dim of q and the pools differ")
    tw = _token_weights(weights, weight_rows, num_new, S, hkv, width * bs, index)
    _run("pa_decode_weights", index, _lib.pa_decode_weights, q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
         block_tables.data_ptr(), width, seq_lens.data_ptr(), S, Hq, scale, out.data_ptr(), ctypes.byref(tw),
         workspace.data_ptr(), ws_bytes, _status_ptr(dev_status, index), _desc_ref(nb, hkv, bs, D, _code(k_pool)),
         _opts_ref(num_ctas, flags), _stream_of(index, stream))


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------


def _want_evict(block_tables, seq_lens, budgets, kept, new_lens, k_pool, v_pool, dst_tables):
    """(device index, pool shape, num_seqs, table width, room of kept) of an eviction."""
    if torch is None:
        _bind()
    try:
        S, width = tables = block_tables.shape
        pool_shape = k_pool.shape
        kept_s, kept_h, room = kept.shape
        index, dtype, i32, one = k_pool.get_device(), k_pool.dtype, torch.int32, (S,)
        if (index >= 0 and (dtype in _codes or (dtype is torch.uint8 and pool_shape[3] in (36, 72))) and kept_s == S
                and kept_h == pool_shape[1] and v_pool.dtype is dtype and v_pool.shape == pool_shape
                and seq_lens.shape == one and budgets.shape == one and new_lens.shape == one
                and block_tables.dtype is i32 and seq_lens.dtype is i32 and budgets.dtype is i32
                and new_lens.dtype is i32 and kept.dtype is i32 and v_pool.get_device() == index
                and block_tables.get_device() == index and seq_lens.get_device() == index
                and budgets.get_device() == index and new_lens.get_device() == index and kept.get_device() == index
                and k_pool.is_contiguous() and v_pool.is_contiguous() and block_tables.is_contiguous()
                and seq_lens.is_contiguous() and budgets.is_contiguous() and new_lens.is_contiguous()
                and kept.is_contiguous()
                and (dst_tables is None or (dst_tables.dtype is i32 and dst_tables.shape == tables
                                            and dst_tables.get_device() == index and dst_tables.is_contiguous()))):
            nb, hkv, bs, row = pool_shape  # four of them
            return index, pool_shape, S, width, room
    except (AttributeError, TypeError, ValueError, IndexError):
        pass
    index = _first(k_pool, "k_pool", 4)
    fp4 = k_pool.dtype is torch.uint8
    index, pool_shape = (_want_fp4_pools if fp4 else _want_16bit_pools)(k_pool, v_pool)
    _want(block_tables, "block_tables", torch.int32, 2, index)
    shape = block_tables.shape
    S, width = shape
    if dst_tables is not None:
        _want(dst_tables, "dst_tables", torch.int32, 2, index)
        if dst_tables.shape != shape:
            raise ValueError("dst_tables must have block_tables' shape")
    _want(seq_lens, "seq_lens", torch.int32, 1, index)
    _want(budgets, "budgets", torch.int32, 1, index)
    _want(new_lens, "new_lens", torch.int32, 1, index)
    if seq_lens.shape[0] != S or budgets.shape[0] != S or new_lens.shape[0] != S:
        raise ValueError("seq_lens, budgets and new_lens must have num_seqs entries")
    _want(kept, "kept", torch.int32, 3, index)
    kept_s, kept_h, room = kept.shape
    if kept_s != S or kept_h != pool_shape[1]:
        raise ValueError("kept must be [num_seqs, num_kv_heads, room]")
    return index, pool_shape, S, width, room


def pa_evict(block_tables, seq_lens, budgets, weights, kept, new_lens, k_pool, v_pool, sinks: int = 0,
             recent: int = 0, dst_tables=None, new_weights=None, weight_rows=None, dev_status=None,
             stream=None, flags: int = 0) -> None:
    """Keep budgets[s] tokens of each sequence (negative: leave it) by their
    accumulated weights, beside its first `sinks` and last `recent` ones, and
    move them together in their order (pa_evict).  Pools are 16-bit, or uint8
    for 4-bit ones.  kept [num_seqs, num_kv_heads, room] int32 and new_lens
    [num_seqs] int32 are written; dst_tables and new_weights are where the
    rows and weights go, in place when None.  flags: 0, or the test hook
    PA_EVICT_TEST_WITHHOLD."""
    index, (nb, hkv, bs, row), S, width, room = _want_evict(block_tables, seq_lens, budgets, kept, new_lens, k_pool,
                                                            v_pool, dst_tables)
    fp4 = k_pool.dtype is torch.uint8
    desc = _desc_ref(nb, hkv, bs, row * 16 // 9, 0) if fp4 else _desc_ref(nb, hkv, bs, row, _code(k_pool))
    tw = _token_weights(weights, weight_rows, 0, S, hkv, width * bs, index)
    if new_weights is not None:
        _want(new_weights, "new_weights", torch.float32, 3, index)
        if new_weights.shape != weights.shape:
            raise ValueError("new_weights must have weights' shape")
    if flags != 0 and flags != PA_EVICT_TEST_WITHHOLD:  # the bits below are not the caller's
        raise PaError(1, "pa_evict")
    _run("pa_evict", index, _lib.pa_evict, block_tables.data_ptr(), _ptr(dst_tables), width, seq_lens.data_ptr(), S,
         budgets.data_ptr(), _int32(sinks, "sinks"), _int32(recent, "recent"), ctypes.byref(tw), _ptr(new_weights),
         kept.data_ptr(), room, new_lens.data_ptr(), fp4 | flags, k_pool.data_ptr(), v_pool.data_ptr(),
         _status_ptr(dev_status, index), desc, _stream_of(index, stream))
