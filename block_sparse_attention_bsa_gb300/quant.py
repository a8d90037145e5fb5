"""Python binding of the calls of include/bsa_quant.h: the paged key/value cache
held in 4 bits.

Argument checks and marshalling only, as in ``paged``, whose conventions hold
here.  A cache is a uint8 tensor of the shape that ``bsa_cache_q4_shape`` gives
(head dim and page size follow from it); K and V have one each.
"""

from __future__ import annotations

import functools
from struct import Struct
from typing import Optional

import torch

from ._lib import load as _load
from .api import _check, _check_buffer, _stream_ptr
from .paged import _BF, _F32, _U8, PAGE_SIZES_SUPPORTED, _check_overlap, _gpu, _ints, _on, _table, _tensor, _wrong

_pack_cache = Struct("7q").pack             # bsaq_cache


def bsa_cache_q4_shape(pages: int, page_size: int, Hkv: int, d: int):
    """Shape ``[pages, Hkv, page_size / 16, 17 d / 2]`` of a uint8 cache of K or of
    V: blocks of 16 slots, 17/64 of the bytes of a bf16 cache."""
    if page_size not in PAGE_SIZES_SUPPORTED:
        raise ValueError(f"page size {page_size} is not supported {PAGE_SIZES_SUPPORTED}")
    if d not in (64, 128):
        raise ValueError(f"head dim {d} is not supported (64 or 128)")
    return int(pages), int(Hkv), page_size // 16, 17 * d // 2


def _cache(t, name: str, index: int):
    """Packed bsaq_cache and the head dim."""
    if isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype is _U8:
        shape = t.shape
        if len(shape) == 4:
            pages, heads, blocks, row = shape
            page, head, block, one = t.stride()
            if row % 17 == 0 and one == 1 and (blocks <= 1 or block == row):
                d = row // 17 * 2
                return _pack_cache(t.data_ptr(), pages, heads, blocks, d, page, head), d
    raise _wrong(t, name, index, "[pages, Hkv, page_size / 16, 17 d / 2] with contiguous blocks", _U8)


def _caches(k_cache, v_cache, index: int):
    kc, d = _cache(k_cache, "k_cache", index)
    return kc, _cache(v_cache, "v_cache", index)[0], d


def bsa_cache_append_q4(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                        page_table: torch.Tensor, kv_lens: torch.Tensor, *, new_lens: Optional[torch.Tensor] = None,
                        stream=None) -> None:
    """Quantises new keys and values ``[B, T, Hkv, d]`` as it writes them into a
    paged cache held in 4 bits (see ``bsa_cache_q4_shape``).

    Positions, lengths and tables are those of ``bsa_cache_append``: token t of
    request b goes to key ``kv_lens[b] - n + t``, n = ``new_lens[b]`` (default T)
    new tokens being counted in ``kv_lens[b]``.  32 neighbouring channels share a
    scale, from 2^-15 to 1.75 2^16; a value is off by at most half of it, which is
    at most 1/13 of the largest of the 32, or 2^-16 where that is more: values below
    2^-16 read as 0 in a group of such.  Above 7 times the largest scale, 802,816,
    they saturate.  A group with a value that is not finite reads as NaN.  Keys
    with rotary positions are rotated before (``bsa_rope_axes``).  A block of 16
    slots that one request's new tokens touch may not be touched by another's.
    """
    dev = _gpu(k, "k")
    kd, vd = _tensor(k, "k", dev), _tensor(v, "v", dev)
    kc, vc, _ = _caches(k_cache, v_cache, dev)
    B = k.shape[0]
    table, stride, n = _table(page_table, B, dev)
    args = (kd, vd, kc, vc, table, stride, n, _ints(kv_lens, "kv_lens", dev, B), _ints(new_lens, "new_lens", dev, B))
    st = _on(dev, stream, _load().bsaq_cache_append, *args)
    if st:
        _check(st)


def bsa_cache_read_q4(k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor,
                      length: int, *, first: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                      v_out: Optional[torch.Tensor] = None, stream=None):
    """Keys and values that a 4-bit cache holds, as bf16 rows ``[B, length, Hkv,
    d]`` for the calls that take rows (``bsa_select``, ``bsa_forward`` ..).

    Row t of request b is key ``first[b] + t`` (int32 ``[B]``; default t), for keys
    below ``kv_lens[b]``; rows behind are not written: zeros in outputs that the
    call makes, what stood there in ``k_out`` and ``v_out`` (any strides with a
    contiguous last dim).  A shared prefix is read as a request of its own:
    ``prefix_table[None]`` with its length.  Returns ``(k, v)``.
    """
    dev = _gpu(k_cache, "k_cache")
    kc, vc, d = _caches(k_cache, v_cache, dev)
    B = page_table.shape[0] if isinstance(page_table, torch.Tensor) and page_table.dim() else -1
    table, stride, n = _table(page_table, B, dev)
    lens, begin = _ints(kv_lens, "kv_lens", dev, B), _ints(first, "first", dev, B)
    shape = (B, int(length), k_cache.shape[1], d)
    if not 0 < shape[1] < 1 << 31:
        raise ValueError(f"length {shape[1]} is out of range")
    kd, vd = _rows_out(k_out, "k_out", shape, dev), _rows_out(v_out, "v_out", shape, dev)
    return _on(dev, stream, _read_launch, (kc, vc, table, stride, n, lens, begin), shape, k_cache.device, k_out, v_out, kd, vd)


def _rows_out(t, name: str, shape, index: int):
    if t is None:
        return None
    packed = _tensor(t, name, index)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape} (got {tuple(t.shape)})")
    return packed


def _read_launch(args, shape, device, k_out, v_out, kd, vd, handle):
    if kd is None:
        k_out = torch.zeros(shape, dtype=_BF, device=device)
        kd = _tensor(k_out, "k_out", device.index)
    if vd is None:
        v_out = torch.zeros(shape, dtype=_BF, device=device)
        vd = _tensor(v_out, "v_out", device.index)
    st = _load().bsaq_cache_read(*args, kd, vd, handle)
    if st:
        _check(st)
    return k_out, v_out


def bsa_forward_paged_q4_workspace_size(B, T, Hq, Hkv, d, has_prefix, num_sms=0) -> int:
    return int(_load().bsaq_forward_workspace_size(B, T, Hq, Hkv, d, 1 if has_prefix else 0, num_sms))


def bsa_forward_paged_q4(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                         kv_lens: torch.Tensor, *, new_lens: Optional[torch.Tensor] = None,
                         prefix_table: Optional[torch.Tensor] = None, prefix_len: int = 0, causal: bool = True,
                         softmax_scale: float = 0.0, out: Optional[torch.Tensor] = None,
                         lse: Optional[torch.Tensor] = None, return_lse: bool = True,
                         workspace: Optional[torch.Tensor] = None, stream=None):
    """``bsa_forward_paged`` over a cache held in 4 bits: attention of T new tokens
    per request (T = 1: one decoding step) to the first ``prefix_len`` keys of the
    pages ``prefix_table``, which all requests share, and to their own keys.

    Arguments, rows, limits and results are those of ``bsa_forward_paged``; the
    caches are those of ``bsa_cache_append_q4``, which is called first.  K and V
    are the values the pages hold, exactly; the softmax's weights are rounded to
    bf16 where they meet V.

    Returns ``(out [B, T, Hq, d] bf16, lse [B, Hq, T] fp32 or None)``.
    """
    prefix_len = int(prefix_len)
    if not 0 <= prefix_len < 1 << 31:          # ctypes would take it modulo 2^32
        raise ValueError(f"prefix_len {prefix_len} is out of range")
    softmax_scale = float(softmax_scale)
    if 0.0 < softmax_scale < 2.0 ** -126:      # as a float it may be 0, which selects d^-1/2
        raise ValueError(f"softmax_scale {softmax_scale} is below the smallest normal float")
    dev = _gpu(q, "q")
    qd = _tensor(q, "q", dev)
    kc, vc, _ = _caches(k_cache, v_cache, dev)
    B = q.shape[0]
    table, stride, n = _table(page_table, B, dev)
    lens, new = _ints(kv_lens, "kv_lens", dev, B), _ints(new_lens, "new_lens", dev, B)
    shared = None
    if prefix_len > 0:
        if prefix_table is None:
            raise ValueError(f"prefix_len is {prefix_len}, prefix_table is None")
        pages = prefix_table.numel() if isinstance(prefix_table, torch.Tensor) else 0
        shared = _ints(prefix_table, "prefix_table", dev, pages)
        if pages * k_cache.shape[2] * 16 < prefix_len:
            raise ValueError(f"prefix_table has {pages} pages of {k_cache.shape[2] * 16}, prefix_len is {prefix_len}")
    return _on(dev, stream, _forward_launch, q, k_cache, v_cache,
               (qd, kc, vc, table, stride, n, lens, new, shared, prefix_len, 1 if causal else 0, softmax_scale),
               out, lse, return_lse, workspace)


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(dev, B, T, Hq, Hkv, d, has_prefix) -> int:
    """What a call on ``dev``, which is current, needs; asking the library takes 2 us."""
    return max(bsa_forward_paged_q4_workspace_size(B, T, Hq, Hkv, d, has_prefix), 256)


def _forward_launch(q, k_cache, v_cache, args, out, lse, return_lse, workspace, handle):
    dev = q.device
    B, T, Hq, d = q.shape
    if out is None:
        out = torch.empty((B, T, Hq, d), dtype=_BF, device=dev)
    else:
        _check_buffer("out", out, (B, T, Hq, d), _BF, dev)
        _check_overlap("out", out, (q, k_cache, v_cache), None)
    if lse is not None:
        _check_buffer("lse", lse, (B, Hq, T), _F32, dev)
    elif return_lse:
        lse = torch.empty((B, Hq, T), dtype=_F32, device=dev)
    if workspace is None:
        workspace = torch.empty(_workspace_bytes(dev, B, T, Hq, k_cache.shape[1], d, args[9] > 0), dtype=_U8, device=dev)
    else:
        _check_buffer("workspace", workspace, (workspace.numel() if isinstance(workspace, torch.Tensor) else 0,), _U8, dev)
    st = _load().bsaq_forward(*args, out.data_ptr(), None if lse is None else lse.data_ptr(), workspace.data_ptr(),
                              workspace.numel(), handle)
    if st:
        _check(st)
    return out, lse


def bsa_debug_paged_q4_wait_probe(limit_ns: int, stream=None) -> None:
    """``bsa_debug_wait_probe`` for the kernels of the attention over 4-bit pages."""
    _check(_load().bsaq_debug_wait_probe(int(limit_ns), _stream_ptr(stream)))
