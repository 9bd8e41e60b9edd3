"""Refusals of the paged-cache calls, on the host before any launch (CPU)."""
import ctypes

import pytest
import torch

import sparse_attention_token_index_b200 as dsa

BF16, FP32, E4M3 = 0, 1, 2
OK = ctypes.c_void_p(4096)
BIG = 1 << 30


@pytest.fixture(scope="module")
def L():
    return dsa.lib()


def _plan(L, **kw):
    a = dict(lens=OK, new=OK, free=OK, n_free=4, used=OK, B=2, page=16, n_pages=8, max_pages=4, max_tokens=8, table=OK,
             q=OK, slots=OK, pos=OK, lo=OK, uo=OK, ws=OK, wb=BIG)
    a.update(kw)
    return L.dsa_page_plan(a["lens"], a["new"], a["free"], a["n_free"], a["used"], a["B"], a["page"], a["n_pages"],
                           a["max_pages"], a["max_tokens"], a["table"], a["q"], a["slots"], a["pos"], a["lo"], a["uo"],
                           a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,code", [
    ({"lens": None}, -1), ({"used": None}, -1), ({"table": None}, -1), ({"slots": None}, -1), ({"free": None}, -1),
    ({"page": 0}, -1), ({"n_pages": 0}, -1), ({"max_pages": 0}, -1), ({"B": -1}, -1), ({"max_tokens": -1}, -1),
    ({"n_free": -1}, -1), ({"B": (1 << 20) + 1}, -1), ({"max_pages": 1 << 20, "page": 1 << 11}, -2), ({"wb": 64}, -3)])
def test_plan_refusals(L, kw, code):
    assert _plan(L, **kw) == code


def test_empty_calls_need_no_device(L):
    assert _plan(L, B=0, lens=None, new=None, used=None, table=None, ws=None) == 0
    assert L.dsa_page_append(None, None, None, 0, 8, 128, BF16, E4M3, None, None, None, None, 4, 16, 16 * 1024, None, 0,
                             None) == 0
    n = ctypes.c_size_t(0)
    assert L.dsa_attend_paged_workspace_size(0, 0, 1, 32, 8, 128, BF16, BF16, ctypes.byref(n)) == 0 and n.value == 256
    assert _attend(L, B=0, total_q=0, Q=None, K=None, V=None, ws=None) == 0
    assert _attend(L, selected=True, B=3, total_q=0, Q=None, K=None, V=None, ws=None) == 0
    # still checked
    assert _attend(L, B=0, total_q=0, Hq=33) == -1


@pytest.mark.parametrize("kw,code", [
    ({"k": None}, -1), ({"slots": None}, -1), ({"K": None}, -1), ({"v": None}, -1), ({"V": None}, -1), ({"ws": None}, -1),
    ({"T": -1}, -1), ({"Hkv": 0}, -1), ({"d": 0}, -1), ({"n_pages": 0}, -1), ({"page": 0}, -1), ({"d": 257}, -2),
    ({"stride": 16 * 8 * 128 - 1}, -1), ({"src": E4M3}, -2), ({"kv": FP32}, -2), ({"ks": OK}, -1),
    ({"kv": E4M3}, -1), ({"kv": E4M3, "ks": OK}, -1), ({"kv": E4M3, "vs": OK}, -1), ({"k": ctypes.c_void_p(4104)}, -1),
    ({"V": ctypes.c_void_p(4097)}, -1), ({"wb": 8}, -3)])
def test_append_refusals(L, kw, code):
    a = dict(k=OK, v=OK, slots=OK, T=4, Hkv=8, d=128, src=BF16, kv=BF16, K=OK, V=OK, ks=None, vs=None, n_pages=4,
             page=16, stride=16 * 8 * 128, ws=OK, wb=256)
    a.update(kw)
    assert L.dsa_page_append(a["k"], a["v"], a["slots"], a["T"], a["Hkv"], a["d"], a["src"], a["kv"], a["K"], a["V"],
                             a["ks"], a["vs"], a["n_pages"], a["page"], a["stride"], a["ws"], a["wb"], None) == code


def _attend(L, selected=False, **kw):
    a = dict(Q=OK, K=OK, V=OK, ks=None, vs=None, table=OK, lens=OK, q=OK, idx=OK, k=16, B=2, total_q=2, max_q=1,
             n_pages=8, page=16, stride=16 * 8 * 128, max_pages=4, Hq=32, Hkv=8, d=128, scale=None, qt=BF16, kv=BF16,
             out=OK, lse=None, ws=OK, wb=BIG)
    a.update(kw)
    head = (a["Q"], a["K"], a["V"], a["ks"], a["vs"], a["table"], a["lens"], a["q"])
    tail = (a["n_pages"], a["page"], a["stride"], a["max_pages"], a["Hq"], a["Hkv"], a["d"], a["scale"], a["qt"],
            a["kv"], a["out"], a["lse"], a["ws"], a["wb"], None)
    if selected:
        return L.dsa_attend_selected(*head, a["idx"], a["k"], a["B"], a["total_q"], *tail)
    return L.dsa_attend_paged(*head, a["B"], a["total_q"], a["max_q"], *tail)


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("kw,code", [
    ({"Q": None}, -1), ({"K": None}, -1), ({"V": None}, -1), ({"table": None}, -1), ({"lens": None}, -1),
    ({"q": None}, -1), ({"out": None}, -1), ({"ws": None}, -1), ({"B": -1}, -1), ({"total_q": -1}, -1),
    ({"page": 0}, -1), ({"n_pages": 0}, -1), ({"max_pages": 0}, -1), ({"stride": 16 * 8 * 128 - 8}, -1),
    ({"Hq": 33}, -1), ({"Hkv": 0}, -1), ({"Hq": 2048}, -2), ({"Hq": 1024, "Hkv": 4, "stride": 1 << 20}, -2),
    ({"d": 257, "stride": 1 << 20}, -2), ({"qt": FP32}, -2), ({"kv": FP32}, -2), ({"qt": E4M3}, -2),
    ({"kv": E4M3}, -1), ({"ks": OK}, -1), ({"vs": OK}, -1), ({"kv": E4M3, "ks": OK}, -1),
    ({"Q": ctypes.c_void_p(4104)}, -1), ({"K": ctypes.c_void_p(4097)}, -1), ({"out": ctypes.c_void_p(4104)}, -1),
    ({"max_pages": 1 << 28}, -2), ({"scale": ctypes.byref(ctypes.c_float(float("nan")))}, -1),
    ({"scale": ctypes.byref(ctypes.c_float(float("inf")))}, -1)])
def test_attend_refusals(L, selected, kw, code):
    assert _attend(L, selected, **kw) == code


def test_attend_size_refusals(L):
    assert _attend(L, max_q=0) == -1 and _attend(L, max_q=65537) == -1
    assert _attend(L, True, k=0) == -1 and _attend(L, True, k=65537) == -1 and _attend(L, True, idx=None) == -1
    assert L.dsa_attend_paged_workspace_size(1, 1, 1, 32, 8, 128, BF16, BF16, None) == -1
    assert L.dsa_status_string(-8) == b"not enough free pages"


def _cpu():
    i32 = dict(dtype=torch.int32)
    return dict(Q=torch.zeros((2, 8, 64), dtype=torch.bfloat16), K=torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16),
                table=torch.zeros((2, 2), **i32), lens=torch.zeros(2, **i32), q=torch.zeros(3, **i32),
                idx=torch.zeros((2, 8), **i32))


def test_binding_refuses_host_tensors_and_bad_shapes():
    # every check that needs no device: shapes and types first, then the place
    t = _cpu()
    with pytest.raises(ValueError):
        dsa.dsa_attend_paged(t["Q"], t["K"], t["K"], t["table"], t["lens"], t["q"], 1)
    with pytest.raises(ValueError):
        dsa.dsa_attend_selected(t["Q"], t["K"], t["K"], t["table"], t["lens"], t["q"], t["idx"])
    with pytest.raises(ValueError):
        dsa.dsa_attend_paged(t["Q"][0], t["K"], t["K"], t["table"], t["lens"], t["q"], 1)
    with pytest.raises(TypeError):
        dsa.dsa_attend_paged(t["Q"].half(), t["K"], t["K"], t["table"], t["lens"], t["q"], 1)
    with pytest.raises(ValueError):
        dsa.dsa_page_append(t["Q"], t["K"], torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        dsa.dsa_page_plan(t["lens"], t["lens"], t["table"], t["lens"], t["lens"][:1], 16, 4, 8)
    with pytest.raises(TypeError):
        dsa.dsa_page_plan(t["lens"].long(), t["lens"], t["table"], t["lens"], t["lens"][:1], 16, 4, 8)


def test_the_extension_takes_no_cpu_tensors():
    ext = dsa._paged._ext()
    i = torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(4096, dtype=torch.uint8)
    assert ext.page_plan(i, i, torch.zeros((2, 4), dtype=torch.int32), i, i[:1], 16, 4, 8, ws) is None
    k = torch.zeros((2, 2, 64))
    assert ext.page_append(k, torch.zeros((1, 4, 2, 64)), i.long(), None, None, None, None, ws) is None
    assert ext.attend(k, torch.zeros((1, 4, 2, 64)), torch.zeros((1, 4, 2, 64)), i[None], i[:1], i, None, None, None, ws, 1,
                      None, True) is None
    for f in (ext.page_plan, ext.page_append, ext.attend):
        assert f() is None and f(1, 2) is None
    with pytest.raises(TypeError):
        ext.bind(1)
