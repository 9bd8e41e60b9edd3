"""Calls of the paged cache that the host refuses or answers without a device:
what would fault, be cut short or be answered wrongly further on (CPU)."""
import ctypes

import pytest
import torch

import sparse_attention_token_index_b200 as dsa
from test_paged_api import BF16, E4M3, OK, _attend, _cpu, _plan


@pytest.fixture(scope="module")
def L():
    return dsa.lib()


def at(offset):
    return ctypes.c_void_p(4096 + offset)


# ---------------------------------------------------------------------------
# addresses
# ---------------------------------------------------------------------------
def _append(L, **kw):
    a = dict(k=OK, v=OK, slots=OK, T=4, Hkv=8, d=128, src=BF16, kv=BF16, K=OK, V=OK, ks=None, vs=None, n_pages=4,
             page=16, stride=16 * 8 * 128, ws=OK, wb=256)
    a.update(kw)
    return L.dsa_page_append(a["k"], a["v"], a["slots"], a["T"], a["Hkv"], a["d"], a["src"], a["kv"], a["K"], a["V"],
                             a["ks"], a["vs"], a["n_pages"], a["page"], a["stride"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("name,offset", [("ws", 1), ("ws", 8), ("slots", 4), ("lens", 2), ("new", 1), ("free", 2), ("used", 2),
                                         ("table", 1), ("q", 2), ("pos", 2), ("lo", 2), ("uo", 3)])
def test_plan_refuses_addresses_off_their_element(L, name, offset):
    assert _plan(L, **{name: at(offset)}) == -1


@pytest.mark.parametrize("name,offset", [("ws", 1), ("ws", 8), ("slots", 4), ("k", 8), ("v", 2), ("K", 1), ("V", 1), ("ks", 2),
                                         ("vs", 1)])
def test_append_refuses_addresses_off_their_element(L, name, offset):
    scaled = dict(kv=E4M3, ks=OK, vs=OK) if name in ("ks", "vs") else {}
    assert _append(L, **{**scaled, name: at(offset)}) == -1


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("name,offset", [("ws", 1), ("ws", 8), ("table", 2), ("lens", 1), ("q", 2), ("idx", 2), ("lse", 2), ("ks", 2),
                                         ("vs", 1), ("Q", 8), ("out", 8), ("K", 1)])
def test_attention_refuses_addresses_off_their_element(L, selected, name, offset):
    if name == "idx" and not selected:
        return
    scaled = dict(kv=E4M3, ks=OK, vs=OK) if name in ("ks", "vs") else {}
    assert _attend(L, selected, **{**scaled, name: at(offset)}) == -1


# ---------------------------------------------------------------------------
# sizes
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("selected", [False, True])
def test_attention_refuses_tables_whose_last_tiles_pass_31_bits(L, selected):
    # a length within a tile of 2^31 overflows where it is rounded up to tiles, or stepped over
    for page, width in (((1 << 31) - 1, 1), (1, (1 << 31) - 8), (1 << 10, 1 << 21), ((1 << 31) - 1023, 1)):
        kw = dict(page=page, max_pages=width, Hq=1, Hkv=1, d=8, stride=page * 8)
        assert _attend(L, selected, **kw) == -2, (page, width)
    # the largest that is taken goes on to the next check
    assert _attend(L, selected, page=(1 << 31) - 1024, max_pages=1, Hq=1, Hkv=1, d=8, stride=((1 << 31) - 1024) * 8, Q=None) == -1
    assert _attend(L, selected, page=1 << 20, max_pages=(1 << 11) - 1, Hq=1, Hkv=1, d=8, stride=8 << 20, Q=None) == -1


@pytest.mark.parametrize("workspace", [None, torch.zeros(4096, dtype=torch.uint8)])
@pytest.mark.parametrize("kw", [{"page": (1 << 32) + 16}, {"n_pages": (1 << 32) + 4}, {"max_tokens": (1 << 32) + 8}, {"page": 16 - (1 << 32)}])
def test_plan_refuses_sizes_beyond_32_bits(workspace, kw):
    t = _cpu()
    a = {"page": 16, "n_pages": 4, "max_tokens": 8, **kw}
    with pytest.raises(ValueError, match="32 bits"):
        dsa.dsa_page_plan(t["lens"], t["lens"], t["table"], t["lens"], t["lens"][:1], workspace=workspace, **a)


def test_other_calls_refuse_sizes_beyond_32_bits():
    t, meta = _cpu(), dict(dtype=torch.bfloat16, device="meta")
    many = torch.empty(((1 << 32) + 4, 16, 2, 64), **meta)
    for call in (lambda: dsa.dsa_attend_paged(t["Q"], t["K"], t["K"], t["table"], t["lens"], t["q"], (1 << 32) + 1),
                 lambda: dsa.dsa_attend_paged(t["Q"], many, many, t["table"], t["lens"], t["q"], 1),
                 lambda: dsa.dsa_attend_selected(t["Q"], many, many, t["table"], t["lens"], t["q"], t["idx"]),
                 lambda: dsa.dsa_page_append(torch.empty(((1 << 32) + 2, 2, 64), **meta), t["K"], t["q"].long()),
                 lambda: dsa.dsa_page_append(t["Q"][:, :2], many, t["lens"].long()),
                 lambda: dsa.page_plan_workspace_bytes(2, (1 << 32) + 8),
                 lambda: dsa._paged._bytes("dsa_attend_paged", None, (1 << 32) + 1, 1, 1, 8, 2, 64, 0, 0)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


# ---------------------------------------------------------------------------
# gradients
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("workspace", [None, torch.zeros(4096, dtype=torch.uint8)])
def test_calls_without_a_backward_pass_refuse_tensors_that_want_a_gradient(workspace):
    t = _cpu()
    for name in ("Q", "K"):
        a = {**t, name: t[name].clone().requires_grad_()}
        for call in (lambda: dsa.dsa_attend_paged(a["Q"], a["K"], a["K"], a["table"], a["lens"], a["q"], 1, workspace=workspace),
                     lambda: dsa.dsa_attend_selected(a["Q"], a["K"], a["K"], a["table"], a["lens"], a["q"], a["idx"],
                                                     workspace=workspace),
                     lambda: dsa.dsa_page_append(a["Q"][:, :2], a["K"], torch.zeros(2, dtype=torch.int64), workspace=workspace)):
            with pytest.raises(RuntimeError, match="gradient"):
                call()
            with torch.no_grad(), pytest.raises(ValueError, match="CUDA|on "):  # the next check
                call()
