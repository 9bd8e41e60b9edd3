"""ctypes binding of the paged-cache calls (``include/dsa_paged.h``; argument marshalling only)."""
from __future__ import annotations

import contextlib
import ctypes
import functools
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


def _need(t: torch.Tensor, what: str, dtype, shape, device=None):
    """`t` is a contiguous CUDA tensor of this dtype and shape (None: any size there)."""
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        raise ValueError(f"{what} must be {list(shape)}, not {list(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{what} must be on a CUDA device (the cache has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{what} is on {t.device}, not {device}")


def _pool(K, V, K_scale, V_scale, device, Hkv=None, d=None) -> Tuple[int, int]:
    """Checks the pages of a cache (V may be absent); (element type, page stride in elements)."""
    code = _type(K, "K_pages", True)
    if K.dim() != 4 or (Hkv is not None and tuple(K.shape[2:]) != (Hkv, d)):
        raise ValueError("K_pages must be [n_pages, page, Hkv, d]" + (f" with Hkv, d = {Hkv}, {d}" if Hkv else ""))
    n, page, hk, dd = K.shape
    stride = K.stride(0) if n > 1 else page * hk * dd
    for t, what in ((K, "K_pages"), (V, "V_pages")):
        if t is None:
            continue
        if not t.is_cuda or t.device != device:
            raise ValueError(f"{what} must be on {device}")
        if t.shape != K.shape or t.dtype != K.dtype:
            raise ValueError(f"{what} must have K_pages' shape and dtype")
        if not t[0].is_contiguous() or (n > 1 and t.stride(0) != stride) or stride < page * hk * dd:
            raise ValueError(f"{what}: the dimensions [page, Hkv, d] must be contiguous, K and V pages equally far apart")
    if (code == DSA_DTYPE_FP8_E4M3) != (K_scale is not None) or \
            (code == DSA_DTYPE_FP8_E4M3 and V is not None) != (V_scale is not None):
        raise ValueError("e4m3 pages (and only they) come with K_scale and V_scale")
    for t, what in ((K_scale, "K_scale"), (V_scale, "V_scale")):
        if t is not None:
            _need(t, what, torch.float32, (n, page, hk), device)
    return code, stride


@contextlib.contextmanager
def _on(device: torch.device, stream):
    """Makes the tensors' device current and yields the stream's handle; what is allocated inside belongs to it."""
    if stream is None:
        if torch.cuda.current_device() == device.index:
            yield torch.cuda.current_stream().cuda_stream
        else:
            with torch.cuda.device(device):
                yield torch.cuda.current_stream().cuda_stream
    else:
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        with torch.cuda.stream(stream):
            yield stream.cuda_stream


def _workspace(nbytes: int, device, workspace):
    if workspace is not None:
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {device}")
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace has {workspace.numel() * workspace.element_size()} bytes, needs {nbytes}")
        return workspace
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


@functools.lru_cache(maxsize=1024)
def _bytes(name: str, device, *args) -> int:
    n = _sz(0)
    with torch.cuda.device(device) if device is not None else contextlib.nullcontext():
        _check(getattr(lib(), name)(*args, ctypes.byref(n)), name)
    return int(n.value)


def page_plan_workspace_bytes(B, max_tokens) -> int:
    return _bytes("dsa_page_plan_workspace_size", None, B, max_tokens)


def attend_paged_workspace_bytes(B, total_q, max_q, Hq, Hkv, d, q_dtype, kv_dtype) -> int:
    return _bytes("dsa_attend_paged_workspace_size", torch.cuda.current_device(), B, total_q, max_q, Hq, Hkv, d,
                  q_dtype, kv_dtype)


def attend_selected_workspace_bytes(B, total_q, k, Hq, Hkv, d, q_dtype, kv_dtype) -> int:
    return _bytes("dsa_attend_selected_workspace_size", torch.cuda.current_device(), B, total_q, k, Hq, Hkv, d,
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
    dev = lens.device
    B = lens.shape[0] if lens.dim() == 1 else -1
    _need(lens, "lens", torch.int32, (B,))
    _need(new_lens, "new_lens", torch.int32, (B,), dev)
    _need(block_table, "block_table", torch.int32, (B, None), dev)
    _need(free_pages, "free_pages", torch.int32, (None,), dev)
    _need(used, "used", torch.int32, (1,), dev)
    max_tokens = int(max_tokens)
    if max_tokens < 0:
        raise ValueError("max_tokens must not be negative")
    with _on(dev, stream) as st:
        if out is None:
            i32 = functools.partial(torch.empty, dtype=torch.int32, device=dev)
            out = (i32(B + 1), torch.empty(max_tokens, dtype=torch.int64, device=dev), i32(max_tokens), i32(B), i32(1))
            if B == 0:  # nothing is launched: the answer of a step without requests
                out[0].zero_(), out[1].fill_(-1), out[2].fill_(-1), out[4].copy_(used)
        else:
            for t, what, dtype, n in zip(out, ("q_offsets", "slots", "positions", "lens_out", "used_out"),
                                         (torch.int32, torch.int64, torch.int32, torch.int32, torch.int32),
                                         (B + 1, max_tokens, max_tokens, B, 1)):
                _need(t, what, dtype, (n,), dev)
        ws = _workspace(page_plan_workspace_bytes(B, max_tokens), dev, workspace)
        q_offsets, slots, positions, lens_out, used_out = out
        _check(lib().dsa_page_plan(_p(lens), _p(new_lens), _p(free_pages), free_pages.numel(), _p(used), B, int(page),
                                   int(n_pages), block_table.shape[1], max_tokens, _p(block_table), _p(q_offsets),
                                   _p(slots), _p(positions), _p(lens_out), _p(used_out), _p(ws),
                                   ws.numel() * ws.element_size(), st), "dsa_page_plan")
        if check:
            _check(lib().dsa_check_status(_p(ws), st), "device status")
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
    if k.dim() != 3:
        raise ValueError("k must be [T, Hkv, d]")
    dev, (T, Hkv, d) = k.device, k.shape
    sd = _type(k, "k", False)
    _need(k, "k", k.dtype, (T, Hkv, d))
    if (v is None) != (V_pages is None):
        raise ValueError("v and V_pages come together")
    if v is not None:
        _need(v, "v", k.dtype, (T, Hkv, d), dev)
    _need(slots, "slots", torch.int64, (T,), dev)
    kd, stride = _pool(K_pages, V_pages, K_scale, V_scale, dev, Hkv, d)
    with _on(dev, stream) as st:
        ws = _workspace(256, dev, workspace)
        _check(lib().dsa_page_append(_p(k), _p(v), _p(slots), T, Hkv, d, sd, kd, _p(K_pages), _p(V_pages),
                                     _p(K_scale), _p(V_scale), K_pages.shape[0], K_pages.shape[1], stride, _p(ws),
                                     ws.numel() * ws.element_size(), st), "dsa_page_append")
        if check:
            _check(lib().dsa_check_status(_p(ws), st), "device status")


def _attend(name, Q, K, V, block_table, lens, q_offsets, idx, max_q, scale, K_scale, V_scale, out, lse, workspace,
            stream, check):
    if Q.dim() != 3 or K.dim() != 4:
        raise ValueError("Q must be [total_q, Hq, d], K_pages [n_pages, page, Hkv, d]")
    dev, (rows, Hq, d) = Q.device, Q.shape
    n_pages, page, Hkv, _ = K.shape
    qd = _type(Q, "Q", False)
    _need(Q, "Q", Q.dtype, (rows, Hq, d))
    kd, stride = _pool(K, V, K_scale, V_scale, dev, Hkv, d)
    B = lens.shape[0] if lens.dim() == 1 else -1
    _need(lens, "lens", torch.int32, (B,), dev)
    _need(q_offsets, "q_offsets", torch.int32, (B + 1,), dev)
    _need(block_table, "block_table", torch.int32, (B, None), dev)
    if idx is not None:
        _need(idx, "idx", torch.int32, (rows, None), dev)
    sc = None if scale is None else ctypes.byref(ctypes.c_float(scale))
    with _on(dev, stream) as st:
        if out is None:
            out = torch.empty_like(Q)
        else:
            _need(out, "out", Q.dtype, (rows, Hq, d), dev)
        if lse is True:
            lse = torch.empty((rows, Hq), dtype=torch.float32, device=dev)
        elif lse is not None:
            _need(lse, "lse", torch.float32, (rows, Hq), dev)
        mid = max_q if idx is None else idx.shape[1]
        ws = _workspace(_bytes(name + "_workspace_size", dev.index, B, rows, mid, Hq, Hkv, d, qd, kd), dev, workspace)
        head = (_p(Q), _p(K), _p(V), _p(K_scale), _p(V_scale), _p(block_table), _p(lens), _p(q_offsets))
        tail = (n_pages, page, stride, block_table.shape[1], Hq, Hkv, d, sc, qd, kd, _p(out), _p(lse), _p(ws),
                ws.numel() * ws.element_size(), st)
        if idx is None:
            r = lib().dsa_attend_paged(*head, B, rows, max_q, *tail)
        else:
            r = lib().dsa_attend_selected(*head, _p(idx), idx.shape[1], B, rows, *tail)
        _check(r, name)
        if check:
            _check(lib().dsa_check_status(_p(ws), st), "device status")
    return out if lse is None else (out, lse)


def dsa_attend_paged(Q: torch.Tensor, K_pages: torch.Tensor, V_pages: torch.Tensor, block_table: torch.Tensor,
                     lens: torch.Tensor, q_offsets: torch.Tensor, max_q: int, scale: Optional[float] = None,
                     K_scale=None, V_scale=None, out=None, return_lse: bool = False, lse=None, workspace=None,
                     stream=None, check: bool = False):
    """Attention of new queries over every cached token.

    Q [total_q, Hq, d] bf16/fp32; pages [n_pages, page, Hkv, d] of the same
    type, or e4m3 with scales [n_pages, page, Hkv]; block_table [B, max_pages],
    lens [B] (new tokens included), q_offsets [B+1], all int32 on the device.
    Request b's m_b <= ``max_q`` query rows sit at its last m_b positions and
    see the tokens up to their own.  Returns out (Q's shape and type), with
    ``return_lse`` also the log-sum-exp [total_q, Hq] fp32.  A query that sees
    nothing has out 0 and lse -inf; rows behind q_offsets[B] stay as they were.
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
