"""The build: what it makes is known by what it was made against, and builds do not meet."""

import os
import sysconfig

import pytest
import torch

from moe_decode_router_gb300 import build as B
from moe_decode_router_gb300 import flint_moe as F


def test_marshalling_is_named_by_interpreter_and_torch():
    F.load_library()
    path = B.binding_path()
    assert os.path.exists(path) and B.up_to_date()
    assert torch.__version__ in path and path.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


@pytest.mark.parametrize("what", ["torch", "interpreter"])
def test_marshalling_built_against_another_is_not_taken(monkeypatch, what):
    """However new the file is."""
    F.load_library()
    here = B.binding_path()
    if what == "torch":
        monkeypatch.setattr(B, "_torch_version", lambda: "1.0")
    else:
        get = sysconfig.get_config_var
        monkeypatch.setattr(sysconfig, "get_config_var", lambda k: ".cpython-39.so" if k == "EXT_SUFFIX" else get(k))
    assert B.binding_path() != here and not B.up_to_date()


def test_builds_work_in_folders_of_their_own(monkeypatch, tmp_path):
    """No file that one build writes is a file of another; only finished ones are moved into place."""
    seen = []

    def compile_(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        seen.append(out)
        with open(out, "w") as f:
            f.write("built")
        return type("Done", (), dict(returncode=0, stdout="", stderr=""))()

    monkeypatch.setattr(B, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libflint_moe.so"))
    monkeypatch.setattr(B.subprocess, "run", compile_)
    B.build(force=True)
    first = set(seen)
    seen.clear()
    B.build(force=True)
    assert first and not first & set(seen)
    assert sorted(os.listdir(tmp_path)) == sorted([os.path.basename(B.LIB), os.path.basename(B.binding_path())])
