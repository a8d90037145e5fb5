"""Python binding of the calls of include/bsa_paged.h: rotary positions with
several axes, the paged key/value cache, attention of new tokens over it.

Argument checks and marshalling only, as in ``api``.  The names carry the
package's ``bsa_`` prefix; the C entry points are ``bsap_rope_axes``,
``bsap_cache_append`` and ``bsap_forward``.  ``stream`` is a torch stream or a
raw stream handle (default: the current stream of the tensors' device);
outputs and workspaces that a call makes itself are allocated on that stream.
"""

from __future__ import annotations

import contextlib
import functools
from struct import Struct
from typing import Optional, Sequence

import torch

from ._lib import load as _load
from .api import _check, _check_buffer, _stream_ptr

PAGE_SIZES_SUPPORTED = (16, 32, 64, 128, 256)


# A single-token step is a few microseconds of GPU work, so the way into the
# library is kept short: descriptors are packed bytes (laid out as the structs of
# bsa.h and bsa_paged.h; ctypes passes their address), the stream handle is read
# without building a torch.cuda.Stream, and no context manager is entered unless
# another device or stream is asked for.
_pack_tensor = Struct("8q").pack            # bsa_tensor
_pack_positions = Struct("4q").pack         # bsap_positions
_pack_rope = Struct("2q3i4x").pack          # bsap_rope
_BF, _I32, _F64, _F32, _U8 = torch.bfloat16, torch.int32, torch.float64, torch.float32, torch.uint8


def _raw_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _wrong(t, name: str, index: int, what: str, dtype) -> Exception:
    """What to raise for a tensor that is not one of ``dtype`` on GPU ``index``
    (any GPU if that is None)."""
    if not isinstance(t, torch.Tensor):
        return TypeError(f"{name} must be a torch.Tensor")
    if index is None and t.get_device() < 0:
        return ValueError(f"{name} must be a CUDA tensor (got {t.device})")
    if index is not None and t.get_device() != index:
        return ValueError(f"{name} is on {t.device}, the call's first tensor on device {index}")
    if t.dtype is not dtype:
        return ValueError(f"{name} must be {dtype} (got {t.dtype})")
    return ValueError(f"{name} must be {what} (got shape {tuple(t.shape)}, strides {tuple(t.stride())})")


def _tensor(t, name: str, index) -> bytes:
    """Packed bsa_tensor of a 4-D bf16 tensor on GPU ``index``."""
    if isinstance(t, torch.Tensor) and t.get_device() == index and index >= 0 and t.dtype is _BF:
        shape, stride = t.shape, t.stride()
        if len(shape) == 4 and (stride[3] == 1 or shape[3] == 1):
            return _pack_tensor(t.data_ptr(), *shape, *stride[:3])
    raise _wrong(t, name, index if index is None or index >= 0 else None,
                 "4-D [B, S, H, d] with a contiguous last dim", _BF)


def _gpu(t, name: str) -> int:
    """The GPU of a call's first tensor."""
    index = t.get_device() if isinstance(t, torch.Tensor) else -1
    if index < 0:
        raise _wrong(t, name, None, "", _BF)
    return index


def _ints(t, name: str, index: int, n: int) -> Optional[int]:
    """Pointer of an int32 vector of n on the call's GPU (None passes as NULL)."""
    if t is None:
        return None
    if (isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype is _I32 and t.shape == (n,)
            and t.is_contiguous()):
        return t.data_ptr()
    raise _wrong(t, name, index, f"contiguous [{n}]", _I32)


def _positions(t, name: str, index: int, B: int, S: int):
    """Packed bsap_positions of int32 positions [B, S, A] or [S, A] (shared by
    the batch), and A."""
    if isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype is _I32:
        shape, stride = t.shape, t.stride()
        if len(shape) == 2:
            shape, stride = (1, *shape), (0, *stride)
        if len(shape) == 3 and shape[1] == S and (shape[0] == B or shape[0] == 1):
            return _pack_positions(t.data_ptr(), stride[0] if shape[0] > 1 else 0, stride[1] if S > 1 else 0,
                                   stride[2]), shape[2]
    raise _wrong(t, name, index, f"[B, S, axes] or [S, axes] with B = {B}, S = {S}", _I32)


def _rope(inv_freq, axes, n_axes: int, interleaved: bool, index: int) -> bytes:
    for name, t, dtype in (("inv_freq", inv_freq, _F64), ("axes", axes, _I32)):
        if not (isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype is dtype and t.dim() == 1
                and t.is_contiguous()):
            raise _wrong(t, name, index, "contiguous [pairs]", dtype)
    pairs = axes.shape[0]
    if inv_freq.shape[0] != pairs:
        raise ValueError(f"inv_freq has {inv_freq.shape[0]} pairs, axes {pairs}")
    return _pack_rope(inv_freq.data_ptr(), axes.data_ptr(), pairs, n_axes, 1 if interleaved else 0)


def _extent(t: torch.Tensor):
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


def _check_overlap(name: str, out: torch.Tensor, inputs, in_place) -> None:
    """Refuses an output that shares memory with an input, but for ``in_place``
    itself when it is contiguous, starts where the output does and is one input
    only (given as q and as k it would be read and overwritten at once)."""
    lo, hi = _extent(out)
    for t in inputs:
        a, z = _extent(t)
        if lo < z and a < hi:
            if not (t is in_place and a == lo and t.is_contiguous()):
                raise ValueError(f"{name} overlaps an input (in place takes the whole contiguous input)")
            in_place = None


@contextlib.contextmanager
def _elsewhere(index, stream):
    with torch.cuda.device(index):
        if stream is None:
            yield
        else:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), torch.device("cuda", index))
            if stream.device.index != index:
                raise ValueError(f"stream is on {stream.device}, the tensors on device {index}")
            with torch.cuda.stream(stream):
                yield


def _on(index, stream, call, *args):
    """``call(*args, stream handle)`` with the tensors' GPU and the call's
    stream current."""
    if stream is None and index == _current_device():
        return call(*args, _raw_stream(index))
    with _elsewhere(index, stream):
        return call(*args, _raw_stream(index))


def bsa_axis_frequencies(sections: Sequence[int], theta: float = 10000.0, layout: str = "sections", device="cuda"):
    """``(inv_freq, axes)`` device tensors for ``bsa_rope_axes``: pair counts
    per axis in ``sections`` (e.g. time, height, width), n pairs in all.

    ``layout``: ``"sections"`` cuts one spectrum theta^(-p/n) into consecutive
    sections; ``"per_axis"`` gives each axis a spectrum theta^(-i/sections[a])
    of its own; ``"cycled"`` deals the one spectrum's pairs to the axes in
    turn, until an axis has its share.
    """
    sections = [int(x) for x in sections]
    if not 1 <= len(sections) <= 4 or min(sections) < 0 or sum(sections) == 0:
        raise ValueError(f"sections must be 1 to 4 non-negative pair counts (got {sections})")
    n = sum(sections)
    if layout == "cycled":
        left, axes = list(sections), []
        while len(axes) < n:
            for a in range(len(left)):
                if left[a]:
                    left[a] -= 1
                    axes.append(a)
    elif layout in ("sections", "per_axis"):
        axes = [a for a, m in enumerate(sections) for _ in range(m)]
    else:
        raise ValueError(f"layout must be 'sections', 'per_axis' or 'cycled' (got {layout!r})")
    if layout == "per_axis":
        inv = [float(theta) ** (-i / m) for m in sections for i in range(m)]
    else:
        inv = [float(theta) ** (-p / n) for p in range(n)]
    return (torch.tensor(inv, dtype=torch.float64, device=device),
            torch.tensor(axes, dtype=torch.int32, device=device))


def _rope_call(q, k, pos_q, pos_k, inv_freq, axes, interleaved, backward, q_out, k_out, stream, names):
    dev = _gpu(q, names[0])
    qd = _tensor(q, names[0], dev)
    pq, n_axes = _positions(pos_q, "pos_q", dev, q.shape[0], q.shape[1])
    rope = _rope(inv_freq, axes, n_axes, interleaved, dev)
    kd = pk = None
    if k is not None:
        kd = _tensor(k, names[1], dev)
        pk, nk = _positions(pos_k, "pos_k", dev, k.shape[0], k.shape[1])
        if nk != n_axes:
            raise ValueError(f"pos_q has {n_axes} axes, pos_k {nk}")
    elif k_out is not None:
        raise ValueError(f"{names[3]} is given without {names[1]}")
    return _on(dev, stream, _rope_launch, q, k, qd, kd, pq, pk, rope, backward, q_out, k_out, names)


def _rope_launch(q, k, qd, kd, pq, pk, rope, backward, q_out, k_out, names, handle):
    dev = q.device
    inputs = (q,) if k is None else (q, k)
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=_BF, device=dev)
    else:
        _check_buffer(names[2], q_out, q.shape, _BF, dev)
        _check_overlap(names[2], q_out, inputs, q)
    if k is not None:
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=_BF, device=dev)
        else:
            _check_buffer(names[3], k_out, k.shape, _BF, dev)
            _check_overlap(names[3], k_out, (q, k, q_out), k)
    st = _load().bsap_rope_axes(qd, kd, pq, pk, rope, 1 if backward else 0, q_out.data_ptr(),
                                None if k is None else k_out.data_ptr(), handle)
    if st:
        _check(st)
    return q_out, k_out


def bsa_rope_axes(q: torch.Tensor, k: Optional[torch.Tensor], pos_q: torch.Tensor, pos_k: Optional[torch.Tensor],
                  inv_freq: torch.Tensor, axes: torch.Tensor, *, interleaved: bool = False,
                  q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, stream=None):
    """Rotary positions with several axes: pair p of a head's channels is turned
    by ``position[axes[p]] * inv_freq[p]``.  (``bsa_select_rope`` rotates by
    tables of fp32 sines and cosines, halves paired, in the selector's own pass
    over Q and K.)

    q ``[B, S, Hq, d]``, k ``[B2, S2, Hkv, d]`` or None; positions int32 ``[B,
    S, A]`` or ``[S, A]`` (A = 1..4, any strides: a permuted ``[A, B, S]`` is
    fine); ``inv_freq`` fp64 and ``axes`` int32 ``[pairs]`` on the GPU (see
    ``bsa_axis_frequencies``), pairs a multiple of 8, at most d/2.  Pairs are
    channels (p, p + pairs), or (2p, 2p + 1) with ``interleaved``; channels from
    2 * pairs on pass through.  Returns ``(q_out, k_out)``, contiguous, to pass
    to ``bsa_select`` and ``bsa_forward``; in place with ``q_out=q`` when q is
    contiguous.
    """
    return _rope_call(q, k, pos_q, pos_k, inv_freq, axes, interleaved, False, q_out, k_out, stream,
                      ("q", "k", "q_out", "k_out"))


def bsa_rope_axes_backward(dq: torch.Tensor, dk: Optional[torch.Tensor], pos_q: torch.Tensor,
                           pos_k: Optional[torch.Tensor], inv_freq: torch.Tensor, axes: torch.Tensor, *,
                           interleaved: bool = False, dq_out: Optional[torch.Tensor] = None,
                           dk_out: Optional[torch.Tensor] = None, stream=None):
    """Gradients of ``bsa_rope_axes`` with respect to q and k, given those of
    its outputs (as ``bsa_backward`` returns them): the rotation turned back."""
    return _rope_call(dq, dk, pos_q, pos_k, inv_freq, axes, interleaved, True, dq_out, dk_out, stream,
                      ("dq", "dk", "dq_out", "dk_out"))


def _table(t, B: int, index: int):
    if isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype is _I32:
        shape, stride = t.shape, t.stride()
        if len(shape) == 2 and shape[0] == B and (shape[1] <= 1 or stride[1] == 1):
            return t.data_ptr(), stride[0] if B > 1 else shape[1], shape[1]
    raise _wrong(t, "page_table", index, f"[B, max_pages] with B = {B} and a contiguous last dim", _I32)


def bsa_cache_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                     page_table: torch.Tensor, kv_lens: torch.Tensor, *, new_lens: Optional[torch.Tensor] = None,
                     q: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                     inv_freq: Optional[torch.Tensor] = None, axes: Optional[torch.Tensor] = None,
                     interleaved: bool = False, q_out: Optional[torch.Tensor] = None, stream=None):
    """Writes new keys and values ``[B, T, Hkv, d]`` into a paged cache
    ``[pages, page_size, Hkv, d]``, K rotated on the way.

    Token t of request b goes to key position ``kv_lens[b] - n + t``, where
    ``kv_lens`` (int32 ``[B]``) counts the request's keys INCLUDING its n =
    ``new_lens[b]`` (default T) new ones; tokens from n on are not written, and
    nothing else of the cache changes.  ``page_table`` int32 ``[B, max_pages]``:
    request b's pages in order (entries behind its length are not read).
    With ``positions`` (int32 ``[B, T, A]``), ``inv_freq`` and ``axes`` k is
    rotated as by ``bsa_rope_axes``, and so is ``q`` when given (all T rows);
    without them k is copied.  New tokens may not lie inside a cache, nor K and
    V share slots.  Returns the rotated q, or None.
    """
    dev = _gpu(k, "k")
    kd = _tensor(k, "k", dev)
    vd, kc, vc = _tensor(v, "v", dev), _tensor(k_cache, "k_cache", dev), _tensor(v_cache, "v_cache", dev)
    B, T = k.shape[:2]
    table, stride, n = _table(page_table, B, dev)
    lens = _ints(kv_lens, "kv_lens", dev, B)
    new = _ints(new_lens, "new_lens", dev, B)
    rope = pos = qd = None
    if positions is not None:
        pos, n_axes = _positions(positions, "positions", dev, B, T)
        rope = _rope(inv_freq, axes, n_axes, interleaved, dev)
    elif inv_freq is not None or axes is not None or q is not None:
        raise ValueError("inv_freq, axes and q are given without positions")
    if q is not None:
        qd = _tensor(q, "q", dev)
    elif q_out is not None:
        raise ValueError("q_out is given without q")
    return _on(dev, stream, _append_launch, (kd, vd, kc, vc, table, stride, n, lens, new, rope, pos, qd), q, q_out,
               (q, k, v, k_cache, v_cache))


def _append_launch(args, q, q_out, inputs, handle):
    ptr = None
    if q is not None:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=_BF, device=q.device)
        else:
            _check_buffer("q_out", q_out, q.shape, _BF, q.device)
            _check_overlap("q_out", q_out, inputs, q)
        ptr = q_out.data_ptr()
    st = _load().bsap_cache_append(*args, ptr, handle)
    if st:
        _check(st)
    return q_out


def bsa_forward_paged_workspace_size(B, T, Hq, Hkv, d, has_prefix, num_sms=0) -> int:
    return int(_load().bsap_forward_workspace_size(B, T, Hq, Hkv, d, 1 if has_prefix else 0, num_sms))


def bsa_forward_paged(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                      kv_lens: torch.Tensor, *, new_lens: Optional[torch.Tensor] = None,
                      prefix_table: Optional[torch.Tensor] = None, prefix_len: int = 0, causal: bool = True,
                      softmax_scale: float = 0.0, out: Optional[torch.Tensor] = None,
                      lse: Optional[torch.Tensor] = None, return_lse: bool = True,
                      workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of T new tokens per request over a paged cache, the form of
    ``bsa_forward_causal`` for tokens that come later (T = 1: one decoding step).

    q ``[B, T, Hq, d]``; cache, ``page_table``, ``kv_lens`` and ``new_lens`` as
    in ``bsa_cache_append`` (which is called first: ``kv_lens`` includes the new
    tokens).  Row i < n of request b sees the first ``prefix_len`` keys of the
    pages ``prefix_table`` (int32 ``[pages]``), which all requests share, and its
    request's own keys, with ``causal`` only those up to position ``kv_lens[b] -
    n + i``.  With ``prefix_len`` 0 there is no prefix, whatever ``prefix_table``
    is.  Rows from n on, and rows without a key, get output 0 and LSE -inf; a row
    whose scores are not finite gets NaN.  The softmax's weights are rounded to
    bf16 where they meet V.

    The prefix is read once for up to 256 rows (tokens times query heads per KV
    head) of the whole batch, padded ones counted, or with each request's own
    keys where T fills tiles: a request with many new tokens goes into a call of
    its own, apart from those with one.

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
    kc, vc = _tensor(k_cache, "k_cache", dev), _tensor(v_cache, "v_cache", dev)
    B, T, Hq, d = q.shape
    table, stride, n = _table(page_table, B, dev)
    lens = _ints(kv_lens, "kv_lens", dev, B)
    new = _ints(new_lens, "new_lens", dev, B)
    shared = None
    if prefix_len > 0:
        if prefix_table is None:
            raise ValueError(f"prefix_len is {prefix_len}, prefix_table is None")
        shared = _ints(prefix_table, "prefix_table", dev,
                       prefix_table.numel() if isinstance(prefix_table, torch.Tensor) else 0)
        if prefix_table.numel() * k_cache.shape[1] < prefix_len:
            raise ValueError(f"prefix_table has {prefix_table.numel()} pages of {k_cache.shape[1]}, prefix_len is "
                             f"{prefix_len}")
    return _on(dev, stream, _forward_launch, q, k_cache, v_cache,
               (qd, kc, vc, table, stride, n, lens, new, shared, prefix_len, 1 if causal else 0, softmax_scale),
               out, lse, return_lse, workspace)


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(dev, B, T, Hq, Hkv, d, has_prefix) -> int:
    """What a call on ``dev``, which is current, needs; asking the library takes 2 us."""
    return max(bsa_forward_paged_workspace_size(B, T, Hq, Hkv, d, has_prefix), 256)


def _forward_launch(q, k_cache, v_cache, args, out, lse, return_lse, workspace, handle):
    dev = q.device
    B, T, Hq, d = q.shape
    lib = _load()
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
        workspace = torch.empty(_workspace_bytes(dev, B, T, Hq, k_cache.shape[2], d, args[9] > 0), dtype=_U8, device=dev)
    else:
        _check_buffer("workspace", workspace, (workspace.numel() if isinstance(workspace, torch.Tensor) else 0,), _U8, dev)
    st = lib.bsap_forward(*args, out.data_ptr(), None if lse is None else lse.data_ptr(), workspace.data_ptr(),
                          workspace.numel(), handle)
    if st:
        _check(st)
    return out, lse


def bsa_debug_paged_wait_probe(limit_ns: int, stream=None) -> None:
    """``bsa_debug_wait_probe`` for the paged attention's kernels."""
    _check(_load().bsap_debug_wait_probe(int(limit_ns), _stream_ptr(stream)))
