"""The Python extension of the paged calls: what a machine without it still
has, and when it is built (CPU)."""
import subprocess
import sys

import pytest
import torch

import sparse_attention_token_index_b200 as dsa
from sparse_attention_token_index_b200 import build as B
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


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """The compiler commands that a build would run; what they would write goes into a folder of the test's own."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("\n".join(cmd))
        return subprocess.CompletedProcess(cmd, 0, "", "")
    for name in ("LIB", "DEBUG_LIB", "EXT", "BUILD"):
        monkeypatch.setattr(B, name, str(tmp_path / name))
    monkeypatch.setattr(B.subprocess, "run", run)
    return ran


def test_the_library_is_built_first_and_without_the_extension(monkeypatch, commands):
    monkeypatch.setenv("CXX", "the-c++-compiler")
    assert B.build() == B.LIB
    assert commands[-1][0] == "the-c++-compiler" and all(c[0] != "the-c++-compiler" for c in commands[:-1]) and len(commands) > 2
    done = len(commands)
    assert B.build() == B.LIB and len(commands) == done  # up to date

    def fails(force=False):
        raise FileNotFoundError("the-c++-compiler")
    monkeypatch.setattr(B, "build_ext", fails)
    with pytest.warns(RuntimeWarning, match="extension"):
        assert B.build(force=True) == B.LIB
    assert len(commands) > done


def test_the_extension_is_built_anew_for_another_torch(monkeypatch, commands):
    B.build_ext()
    B.build_ext()
    assert len(commands) == 1
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    B.build_ext()
    B.build_ext()
    assert len(commands) == 2
    monkeypatch.setattr(B, "_nvcc", lambda: 1 / 0)  # a binary that fits asks for no compiler
    B.build_ext()


def test_the_extension_says_what_it_was_built_for():
    assert torch.__version__ in dsa._paged._ext().__doc__
