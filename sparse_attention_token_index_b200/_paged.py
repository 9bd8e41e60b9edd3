"""Binding of the paged-cache calls (``include/dsa_paged.h``; argument marshalling only).

A plain call (on the current device and stream, outputs allocated here, with a
workspace) goes through the ``_paged_ext`` extension; every other one, and any
whose arguments do not pass, through the checks below and ctypes.  Both reach
the same library call; where the extension is missing all go the second way.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import warnings
from typing import Optional, Tuple

import torch

from . import _binding as _b
from ._binding import DSA_DTYPE_BF16, DSA_DTYPE_FP32, DSA_DTYPE_FP8_E4M3, _check, lib

_int, _i64, _sz, _vp = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p
_szp, _fp = ctypes.POINTER(_sz), ctypes.POINTER(ctypes.c_float)
_b._SIGS.update({
    "dsa_page_plan_workspace_size": (_int, [_int, _int, _szp]),
    "dsa_page_plan": (_int, [_vp, _vp, _vp, _int, _vp, _int, _int, _int, _int, _int] + [_vp] * 7 + [_sz, _vp]),
    "dsa_page_append": (_int, [_vp, _vp, _vp, _int, _int, _int, _int, _int, _vp, _vp, _vp, _vp, _int, _int, _i64, _vp,
                               _sz, _vp]),
    "dsa_attend_paged_workspace_size": (_int, [_int] * 8 + [_szp]),
    "dsa_attend_paged": (_int, [_vp] * 8 + [_int] * 5 + [_i64] + [_int] * 4 + [_fp, _int, _int, _vp, _vp, _vp, _sz,
                                                                               _vp]),
    "dsa_attend_selected_workspace_size": (_int, [_int] * 8 + [_szp]),
    "dsa_attend_selected": (_int, [_vp] * 9 + [_int] * 5 + [_i64] + [_int] * 4 + [_fp, _int, _int, _vp, _vp, _vp, _sz,
                                                                                  _vp]),
})
EXPORTED_SYMBOLS = ("dsa_page_plan_workspace_size", "dsa_page_plan", "dsa_page_append",
                    "dsa_attend_paged_workspace_size", "dsa_attend_paged", "dsa_attend_selected_workspace_size",
                    "dsa_attend_selected")

_TYPES = {torch.bfloat16: DSA_DTYPE_BF16, torch.float32: DSA_DTYPE_FP32, torch.uint8: DSA_DTYPE_FP8_E4M3,
          torch.float8_e4m3fn: DSA_DTYPE_FP8_E4M3}


def _type(t: torch.Tensor, what: str, fp8: bool) -> int:
    code = _TYPES.get(t.dtype)
    if code is None or (code == DSA_DTYPE_FP8_E4M3 and not fp8):
        raise TypeError(f"{what}: unsupported dtype {t.dtype}")
    return code


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _refuse(t: torch.Tensor, what: str, dtype, shape, device):
    """Says what is wrong with a tensor that `_need` does not take."""
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must be {list(shape)}, not {list(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{what} must be on a CUDA device (the cache has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    raise ValueError(f"{what} is on {t.device}, not {device}")


def _need(t: torch.Tensor, what: str, dtype, shape, device):
    """`t` is a contiguous tensor of this dtype and shape on this CUDA device."""
    if not (t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous() and t.device == device):
        _refuse(t, what, dtype, shape, device)


def _pool(K, V, K_scale, V_scale, device, Hkv, d) -> Tuple[int, int]:
    """Checks the pages of a cache (V may be absent); (element type, page stride in elements)."""
    code = _type(K, "K_pages", True)
    shape = K.shape
    if len(shape) != 4 or shape[2] != Hkv or shape[3] != d:
        raise ValueError(f"K_pages must be [n_pages, page, Hkv, d] with Hkv, d = {Hkv}, {d}")
    n, page = shape[0], shape[1]
    inner = page * Hkv * d
    stride = K.stride(0) if n > 1 else inner
    for t, what in ((K, "K_pages"), (V, "V_pages")):
        if t is None:
            continue
        if not t.is_cuda or t.device != device:
            raise ValueError(f"{what} must be on {device}")
        if t.shape != shape or t.dtype is not K.dtype:
            raise ValueError(f"{what} must have K_pages' shape and dtype")
        if t.is_contiguous() and (n <= 1 or stride == inner):
            continue
        if not t[0].is_contiguous() or (n > 1 and t.stride(0) != stride) or stride < inner:
            raise ValueError(f"{what}: the dimensions [page, Hkv, d] must be contiguous, K and V pages equally far apart")
    fp8 = code == DSA_DTYPE_FP8_E4M3
    if fp8 != (K_scale is not None) or (fp8 and V is not None) != (V_scale is not None):
        raise ValueError("e4m3 pages (and only they) come with K_scale and V_scale")
    if K_scale is not None:
        _need(K_scale, "K_scale", torch.float32, (n, page, Hkv), device)
    if V_scale is not None:
        _need(V_scale, "V_scale", torch.float32, (n, page, Hkv), device)
    return code, stride


def _ints(name: str, *sizes: int) -> None:
    """Sizes that the library takes as 32-bit numbers (ctypes would cut others short without a word)."""
    if max(sizes) > 0x7fffffff or min(sizes) < -0x80000000:
        raise ValueError(f"{name}: a size does not fit 32 bits: {list(sizes)}")


def _no_gradients(name: str, *tensors) -> None:
    """None of the tensors wants a gradient that the call would lose."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise RuntimeError(f"{name} has no backward pass, and a tensor given to it requires a gradient: detach it, or call "
                           "under torch.no_grad()")


_same = contextlib.nullcontext()
_EXT = None


def _ext():
    """The extension, bound to the loaded library; raises if it has not been built."""
    global _EXT
    if not _EXT:
        try:
            from . import _paged_ext
        except ImportError as e:
            raise RuntimeError("the _paged_ext extension is missing or does not fit this torch: build it with "
                               "`python -m sparse_attention_token_index_b200.build`") from e
        L = lib()
        _paged_ext.bind(*(ctypes.cast(getattr(L, n), _vp).value for n in EXPORTED_SYMBOLS))
        _EXT = _paged_ext
    return _EXT


def _plain():
    """The extension for plain calls; None where it cannot be imported (said once)."""
    global _EXT
    if _EXT is None:
        try:
            from . import _paged_ext  # noqa: F401
        except ImportError as e:
            warnings.warn(f"_paged_ext cannot be imported ({e}): paged calls take a few microseconds longer on the host; build it "
                          "with `python -m sparse_attention_token_index_b200.build`", RuntimeWarning, stacklevel=3)
            _EXT = False
        else:
            _ext()
    return _EXT or None


def _on(device: torch.device, stream):
    """(a context that makes the tensors' device and the call's stream current, or None when they are; the stream's
    handle): what is allocated inside belongs to that stream."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        return torch.cuda.stream(stream), stream.cuda_stream
    index = device.index
    if torch.cuda.current_device() == index:
        return None, _raw_stream(index)
    return torch.cuda.device(device), torch.cuda.current_stream(device).cuda_stream


def _raw_stream(index: int) -> int:
    """The handle of a device's current stream (torch's accessor for compiled code: 0.1 us, the public one takes 3)."""
    return torch._C._cuda_getCurrentRawStream(index)


def _workspace(nbytes: int, device, workspace):
    if workspace is None:
        return torch.zeros(nbytes, dtype=torch.uint8, device=device), nbytes
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    size = workspace.numel() * workspace.element_size()
    if size < nbytes:
        raise ValueError(f"workspace has {size} bytes, needs {nbytes}")
    return workspace, size


@functools.lru_cache(maxsize=1024)
def _bytes(name: str, device, *args) -> int:
    n = _sz(0)
    _ints(name, *args)
    with torch.cuda.device(device) if device is not None else contextlib.nullcontext():
        _check(getattr(lib(), name + "_workspace_size")(*args, ctypes.byref(n)), name)
    return int(n.value)


def page_plan_workspace_bytes(B, max_tokens) -> int:
    return _bytes("dsa_page_plan", None, B, max_tokens)


def attend_paged_workspace_bytes(B, total_q, max_q, Hq, Hkv, d, q_dtype, kv_dtype) -> int:
    return _bytes("dsa_attend_paged", torch.cuda.current_device(), B, total_q, max_q, Hq, Hkv, d,
                  q_dtype, kv_dtype)


def attend_selected_workspace_bytes(B, total_q, k, Hq, Hkv, d, q_dtype, kv_dtype) -> int:
    return _bytes("dsa_attend_selected", torch.cuda.current_device(), B, total_q, k, Hq, Hkv, d,
                  q_dtype, kv_dtype)


def dsa_page_plan(lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                  used: torch.Tensor, page: int, n_pages: int, max_tokens: int, out=None, workspace=None, stream=None,
                  check: bool = False):
    """Block tables and slot maps of one step, from request lengths.

    lens, new_lens [B] int32: tokens each request holds and adds; block_table
    [B, max_pages] int32 is updated in place with pages taken, in order, from
    ``free_pages`` behind the first ``used`` [1] ones.  Returns (q_offsets
    [B+1] int32, slots [max_tokens] int64, positions [max_tokens] int32,
    lens_out [B] int32, used_out [1] int32); ``out`` takes the five
    preallocated, of which lens_out and used_out may be ``lens`` and ``used``
    themselves.  Slots and positions behind the last new token are -1.  Too
    few free pages (DSA_ERR_PAGES) or lengths out of range fail as a whole:
    the table stays, the step has no tokens, and the status word tells.
    """
    if out is None and stream is None and not check and workspace is not None and (ext := _EXT or _plain()):
        r = ext.page_plan(lens, new_lens, block_table, free_pages, used, page, n_pages, max_tokens, workspace)
        if r is not None:
            return r if type(r) is tuple else _check(r, "dsa_page_plan")
    dev = lens.device
    if lens.dim() != 1 or block_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("lens must be [B], block_table [B, max_pages], free_pages [n_free]")
    B, i32 = lens.shape[0], torch.int32
    width, n_free, max_tokens = block_table.shape[1], free_pages.shape[0], int(max_tokens)
    _ints("dsa_page_plan", B, width, n_free, int(page), int(n_pages), max_tokens)
    _need(lens, "lens", i32, (B,), dev)
    _need(new_lens, "new_lens", i32, (B,), dev)
    _need(block_table, "block_table", i32, (B, width), dev)
    _need(free_pages, "free_pages", i32, (n_free,), dev)
    _need(used, "used", i32, (1,), dev)
    if max_tokens < 0:
        raise ValueError("max_tokens must not be negative")
    context, st = _on(dev, stream)
    with context or _same:
        i64, empty = torch.int64, torch.empty
        if out is None:
            out = (empty(B + 1, dtype=i32, device=dev), empty(max_tokens, dtype=i64, device=dev),
                   empty(max_tokens, dtype=i32, device=dev), empty(B, dtype=i32, device=dev),
                   empty(1, dtype=i32, device=dev))
        else:
            for t, what, dtype, n in zip(out, ("q_offsets", "slots", "positions", "lens_out", "used_out"),
                                         (i32, i64, i32, i32, i32), (B + 1, max_tokens, max_tokens, B, 1)):
                _need(t, what, dtype, (n,), dev)
        ws, size = _workspace(page_plan_workspace_bytes(B, max_tokens), dev, workspace)
        q_offsets, slots, positions, lens_out, used_out = out
        r = lib().dsa_page_plan(lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(), n_free, used.data_ptr(), B,
                                int(page), int(n_pages), width, max_tokens, block_table.data_ptr(), q_offsets.data_ptr(),
                                slots.data_ptr(), positions.data_ptr(), lens_out.data_ptr(), used_out.data_ptr(),
                                ws.data_ptr(), size, st)
        if r:
            _check(r, "dsa_page_plan")
        if B == 0:  # nothing is launched: the answer of a step without requests
            out[0].zero_(), out[1].fill_(-1), out[2].fill_(-1), out[4].copy_(used)
        if check:
            _check(lib().dsa_check_status(ws.data_ptr(), st), "device status")
    return out


def dsa_page_append(k: torch.Tensor, K_pages: torch.Tensor, slots: torch.Tensor, v: Optional[torch.Tensor] = None,
                    V_pages: Optional[torch.Tensor] = None, K_scale: Optional[torch.Tensor] = None,
                    V_scale: Optional[torch.Tensor] = None, workspace=None, stream=None, check: bool = False) -> None:
    """Writes rows k (and v) [T, Hkv, d] into their cache slots [T] int64.

    Negative slots skip their row.  The pages [n_pages, page, Hkv, d] have the
    rows' type, or are e4m3 with fp32 scales [n_pages, page, Hkv], one for
    each token and head: scale = max(amax / 448, 2^-126).  ``v`` and
    ``V_pages`` may be left out (a cache of keys alone).
    """
    if stream is None and not check and workspace is not None and (ext := _EXT or _plain()):
        r = ext.page_append(k, K_pages, slots, v, V_pages, K_scale, V_scale, workspace)
        if r is not None:
            return _check(r, "dsa_page_append")
    if k.dim() != 3:
        raise ValueError("k must be [T, Hkv, d]")
    _no_gradients("dsa_page_append", k, v, K_pages, V_pages)
    dev, shape = k.device, k.shape
    T, Hkv, d = shape
    _ints("dsa_page_append", *shape, *K_pages.shape)
    sd = _type(k, "k", False)
    _need(k, "k", k.dtype, shape, dev)
    if (v is None) != (V_pages is None):
        raise ValueError("v and V_pages come together")
    if v is not None:
        _need(v, "v", k.dtype, shape, dev)
    _need(slots, "slots", torch.int64, (T,), dev)
    kd, stride = _pool(K_pages, V_pages, K_scale, V_scale, dev, Hkv, d)
    n_pages, page = K_pages.shape[:2]
    context, st = _on(dev, stream)
    with context or _same:
        ws, size = _workspace(256, dev, workspace)
        r = lib().dsa_page_append(k.data_ptr(), _p(v), slots.data_ptr(), T, Hkv, d, sd, kd, K_pages.data_ptr(),
                                  _p(V_pages), _p(K_scale), _p(V_scale), n_pages, page, stride, ws.data_ptr(), size, st)
        if r:
            _check(r, "dsa_page_append")
        if check:
            _check(lib().dsa_check_status(ws.data_ptr(), st), "device status")


def _attend(name, Q, K, V, block_table, lens, q_offsets, idx, max_q, scale, K_scale, V_scale, out, lse, workspace,
            stream, check):
    if out is None and stream is None and not check and workspace is not None and (lse is None or lse is True) \
            and (ext := _EXT or _plain()):
        r = ext.attend(Q, K, V, block_table, lens, q_offsets, idx, K_scale, V_scale, workspace, max_q, scale, lse is True)
        if r is not None:
            return _check(r, name) if type(r) is int else r
    if Q.dim() != 3 or K.dim() != 4 or lens.dim() != 1 or block_table.dim() != 2 or (idx is not None and idx.dim() != 2):
        raise ValueError("Q must be [total_q, Hq, d], K_pages [n_pages, page, Hkv, d], lens [B], block_table "
                         "[B, max_pages], idx [total_q, k]")
    _no_gradients(name, Q, K, V, K_scale, V_scale)
    dev, dtype, shape, i32 = Q.device, Q.dtype, Q.shape, torch.int32
    rows, Hq, d = shape
    n_pages, page, Hkv, _ = K.shape
    _ints(name, *shape, *K.shape, *lens.shape, *block_table.shape, max_q, *(() if idx is None else idx.shape))
    qd = _type(Q, "Q", False)
    _need(Q, "Q", dtype, shape, dev)
    kd, stride = _pool(K, V, K_scale, V_scale, dev, Hkv, d)
    B, width = lens.shape[0], block_table.shape[1]
    _need(lens, "lens", i32, (B,), dev)
    _need(q_offsets, "q_offsets", i32, (B + 1,), dev)
    _need(block_table, "block_table", i32, (B, width), dev)
    k = max_q
    if idx is not None:
        k = idx.shape[1]
        _need(idx, "idx", i32, (rows, k), dev)
    sc = None if scale is None else ctypes.byref(ctypes.c_float(scale))
    context, st = _on(dev, stream)
    with context or _same:
        if out is None:
            out = torch.empty_like(Q)
        else:
            _need(out, "out", dtype, shape, dev)
        if lse is True:
            lse = torch.empty((rows, Hq), dtype=torch.float32, device=dev)
        elif lse is not None:
            _need(lse, "lse", torch.float32, (rows, Hq), dev)
        ws, size = _workspace(_bytes(name, dev.index, B, rows, k, Hq, Hkv, d, qd, kd), dev, workspace)
        L = lib()
        if idx is None:
            r = L.dsa_attend_paged(Q.data_ptr(), K.data_ptr(), V.data_ptr(), _p(K_scale), _p(V_scale),
                                   block_table.data_ptr(), lens.data_ptr(), q_offsets.data_ptr(), B, rows, max_q,
                                   n_pages, page, stride, width, Hq, Hkv, d, sc, qd, kd, out.data_ptr(), _p(lse),
                                   ws.data_ptr(), size, st)
        else:
            r = L.dsa_attend_selected(Q.data_ptr(), K.data_ptr(), V.data_ptr(), _p(K_scale), _p(V_scale),
                                      block_table.data_ptr(), lens.data_ptr(), q_offsets.data_ptr(), idx.data_ptr(), k,
                                      B, rows, n_pages, page, stride, width, Hq, Hkv, d, sc, qd, kd, out.data_ptr(),
                                      _p(lse), ws.data_ptr(), size, st)
        if r:
            _check(r, name)
        if check:
            _check(L.dsa_check_status(ws.data_ptr(), st), "device status")
    return out if lse is None else (out, lse)


def dsa_attend_paged(Q: torch.Tensor, K_pages: torch.Tensor, V_pages: torch.Tensor, block_table: torch.Tensor,
                     lens: torch.Tensor, q_offsets: torch.Tensor, max_q: int, scale: Optional[float] = None,
                     K_scale=None, V_scale=None, out=None, return_lse: bool = False, lse=None, workspace=None,
                     stream=None, check: bool = False):
    """Attention of new queries over every cached token.

    Q [total_q, Hq, d] bf16/fp32; pages [n_pages, page, Hkv, d] of the same
    type, or e4m3 with scales [n_pages, page, Hkv]; none of them may require a
    gradient (there is no backward pass); block_table [B, max_pages],
    lens [B] (new tokens included), q_offsets [B+1], all int32 on the device.
    Request b's m_b <= ``max_q`` query rows sit at its last m_b positions and
    see the tokens up to their own.  Returns out (Q's shape and type), with
    ``return_lse`` also the log-sum-exp [total_q, Hq] fp32.  A query that sees
    nothing has out 0 and lse -inf; rows in front of q_offsets[0] and from
    q_offsets[B] on are not written: they stay as they were in ``out`` and
    ``lse``, and are not set in outputs that are allocated here.
    """
    return _attend("dsa_attend_paged", Q, K_pages, V_pages, block_table, lens, q_offsets, None, int(max_q), scale,
                   K_scale, V_scale, out, True if return_lse and lse is None else lse, workspace, stream, check)


def dsa_attend_selected(Q: torch.Tensor, K_pages: torch.Tensor, V_pages: torch.Tensor, block_table: torch.Tensor,
                        lens: torch.Tensor, q_offsets: torch.Tensor, idx: torch.Tensor,
                        scale: Optional[float] = None, K_scale=None, V_scale=None, out=None,
                        return_lse: bool = False, lse=None, workspace=None, stream=None, check: bool = False):
    """Attention of query rows over the positions the indexer chose for them.

    idx [total_q, k] int32, as the ``dsa_index_*`` calls answer it: positions
    local to the row's request; entries below 0 or beyond the row's own
    position are skipped.  All else as for ``dsa_attend_paged``; a request may
    own any number of rows.
    """
    return _attend("dsa_attend_selected", Q, K_pages, V_pages, block_table, lens, q_offsets, idx, 0, scale, K_scale,
                   V_scale, out, True if return_lse and lse is None else lse, workspace, stream, check)
