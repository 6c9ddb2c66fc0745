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


# ------------------------------------------------------------------ without the compiled marshalling


def test_library_builds_without_the_marshalling(monkeypatch, tmp_path):
    """A host compiler that fails costs a warning; the library is built and taken."""
    def compile_(cmd, **kw):
        fails = cmd[0] == "no-such-compiler"
        if not fails:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write("built")
        return type("Done", (), dict(returncode=int(fails), stdout="", stderr="no headers"))()

    monkeypatch.setenv("CXX", "no-such-compiler")
    monkeypatch.setattr(B, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libflint_moe.so"))
    monkeypatch.setattr(B.subprocess, "run", compile_)
    with pytest.warns(RuntimeWarning, match="no headers"):
        assert B.build(force=True) == B.LIB
    assert os.listdir(tmp_path) == ["libflint_moe.so"] and B.library_up_to_date()


@pytest.mark.parametrize("broken", ["absent", "not a module"])
def test_library_loads_without_the_marshalling(monkeypatch, tmp_path, broken):
    F.load_library()
    path = tmp_path / "binding.so"
    if broken != "absent":
        path.write_text("not a module")
    monkeypatch.setattr(F, "_LIB", None)
    monkeypatch.setattr(F, "_FAST", F._NotLoaded())
    monkeypatch.setattr(B, "binding_path", lambda: str(path))
    with pytest.warns(RuntimeWarning, match="could not be loaded"):
        lib = F.load_library(build_if_missing=False)
    assert lib is not None and isinstance(F._FAST, F._NotLoaded)
    with pytest.raises(ValueError, match="current CUDA device"):
        F.route(torch.zeros(4, 64), torch.zeros(4, 6, dtype=torch.int32), torch.zeros(4, 6))


@pytest.mark.gpu
def test_both_marshallings_make_the_same_calls(monkeypatch):
    """Every call through the compiled look and through Python's, rows apart and streams given."""
    F.load_library()
    assert not isinstance(F._FAST, F._NotLoaded)
    d = torch.device("cuda:0")
    g = torch.Generator().manual_seed(3)
    T, E, k, K, N = 40, 24, 3, 272, 264
    logits = torch.randn(T, E + 8, generator=g).to(d)[:, :E]
    bias = (0.1 * torch.randn(E, generator=g)).to(d)
    x = torch.randn(T, 2 * K + 8, generator=g).to(torch.bfloat16).to(d)[:, :2 * K]
    b = torch.randn(E, N, K, generator=g).to(torch.float8_e4m3fn).to(d)
    bs = torch.rand(E, -(-N // 128), -(-K // 128), generator=g).to(d)
    shared = torch.randn(T, N, generator=g).to(torch.bfloat16).to(d)

    def layer(stream):
        i32 = dict(dtype=torch.int32, device=d)
        ids, w = torch.zeros(T, k, **i32), torch.zeros(T, k, device=d)
        offsets, order, pos = torch.zeros(E + 1, **i32), torch.zeros(T * k, **i32), torch.zeros(T, k, **i32)
        q, s = torch.zeros(T * k, K, dtype=torch.float8_e4m3fn, device=d), torch.zeros(-(-K // 128), T * k, device=d)
        y, out = torch.zeros(T * k, N, device=d), torch.zeros(T, N, dtype=torch.bfloat16, device=d)
        torch.cuda.synchronize()
        F.route(logits, ids, w, bias=bias, score=F.SCORE_SOFTMAX, n_groups=4, top_groups=2, group_score=F.GROUP_TOP2,
                renormalise=False, scale=2.5, stream=stream)
        F.group_pairs(ids, offsets, order, pos, stream=stream)
        F.quantize_rows(x, q, s, pos=pos, silu_mul=True, stream=stream)
        F.block_gemm(q, s, b, bs, y, offsets=offsets, stream=stream)
        F.combine(y, pos, w, out, shared=shared, stream=stream)
        torch.cuda.synchronize()
        return ids, w, offsets, order, pos, q.view(torch.uint8), s, y, out

    for stream in (None, torch.cuda.Stream()):
        compiled = layer(stream)
        with monkeypatch.context() as m:
            m.setattr(F, "_FAST", F._NotLoaded())
            plain = layer(stream)
        for a, c in zip(compiled, plain):
            assert torch.equal(a, c)
