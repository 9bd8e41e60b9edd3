"""The Python extension of the paged calls: what a machine without it still
has, and when it is built (CPU)."""
import sys

import pytest
import torch

import sparse_attention_token_index_b200 as dsa
from test_paged_api import _cpu


def _calls(t, ws):
    return [lambda: dsa.dsa_page_plan(t["lens"], t["lens"], t["table"], t["lens"], t["lens"][:1], 16, 4, 8, workspace=ws),
            lambda: dsa.dsa_page_append(t["Q"][:, :2].contiguous(), t["K"], t["lens"].long(), workspace=ws),
            lambda: dsa.dsa_attend_paged(t["Q"], t["K"], t["K"], t["table"], t["lens"], t["q"], 1, workspace=ws),
            lambda: dsa.dsa_attend_selected(t["Q"], t["K"], t["K"], t["table"], t["lens"], t["q"], t["idx"], workspace=ws)]


def test_calls_do_without_the_extension(monkeypatch):
    # the same call with a workspace and without one: both go on to the checks, the first says once why it is slower
    name = dsa.__name__ + "._paged_ext"
    monkeypatch.setattr(dsa._paged, "_EXT", None)
    monkeypatch.delattr(dsa, "_paged_ext", raising=False)
    monkeypatch.setitem(sys.modules, name, None)  # an import of it fails
    ws = torch.zeros(4096, dtype=torch.uint8)
    for i, call in enumerate(_calls(_cpu(), ws)):
        if i == 0:
            with pytest.warns(RuntimeWarning, match="_paged_ext"), pytest.raises(ValueError, match="CUDA"):
                call()
        else:
            with pytest.raises(ValueError, match="CUDA|must be on"):
                call()
    with pytest.raises(RuntimeError, match="build it"):
        dsa._paged._ext()
