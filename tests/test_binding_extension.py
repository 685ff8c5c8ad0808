"""The binding's extension: what works where it is missing, and what it is built for (no GPU)."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "latent_mixture_experts_router_gb300"


@pytest.fixture
def build():
    from conftest import build_library
    build_library()
    import __graft_entry__
    return __graft_entry__._build_module()


def run(code, root):
    return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root,
                          env={**os.environ, "PYTHONPATH": str(root)})


def test_without_the_extension_only_its_calls_are_missing(build, tmp_path):
    pkg = tmp_path / PKG
    pkg.mkdir()
    for f in ("__init__.py", "_lib.py", "build.py"):
        shutil.copy(os.path.join(ROOT, PKG, f), pkg / f)
    os.symlink(build.LIB, pkg / os.path.basename(build.LIB))
    r = run(f"""
import torch, {PKG} as lm
assert lm.__file__.startswith({str(tmp_path)!r})
assert lm.lmoe_kernel_launches() == 0 and lm.lmoe_fp8_padded_rows(100, 2) == 256
x = torch.zeros(8, 64, dtype=torch.bfloat16)
n = torch.zeros(1)
for call in (lambda: lm.lmoe_gated_ffn(x, x, x, x), lambda: lm.lmoe_matmul_bf16(x, x, x),
             lambda: lm._lib._tensors.gradients([x], "grads", 0)):
    try:
        call()
    except ImportError as e:
        assert "__graft_entry__" in str(e), e
    else:
        raise AssertionError("called")
""", tmp_path)
    assert r.returncode == 0, r.stderr


def test_the_library_is_made_where_the_extension_is_not(build, tmp_path, monkeypatch):
    lib = str(tmp_path / "liblatent_moe.so")
    monkeypatch.setattr(build, "LIB", lib)
    monkeypatch.setattr(build, "LIB_TENSORS", str(tmp_path / "_tensors.so"))
    for cmd in (["false"], [str(tmp_path / "no_compiler")]):
        monkeypatch.setattr(build, "_tensors_cmd", lambda src: cmd)
        with pytest.raises(RuntimeError, match="tensors.cpp"):
            build.build()
        assert os.path.exists(lib)
        os.remove(lib)


def test_the_extension_is_made_again_for_another_torch(build, tmp_path, monkeypatch):
    """As after an upgrade: the source is as old as it was, torch is not."""
    made = []

    def fake(cmd, **kw):
        made.append(cmd)
        if "-o" in cmd:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")
    root, version = build._torch()
    monkeypatch.setattr(build, "LIB_TENSORS", str(tmp_path / "_tensors.so"))
    monkeypatch.setattr(build.subprocess, "run", fake)
    for v, commands in ((version, 1), (version, 1), ("1.0+other", 2), ("1.0+other", 2), (version, 3)):
        monkeypatch.setattr(build, "_torch", lambda: (root, v))
        build.build()
        assert len(made) == commands and all(any("tensors.cpp" in a for a in c) for c in made)
    monkeypatch.setenv("CXX", "another-compiler")
    build.build()
    assert len(made) == 4 and made[-1][0] == "another-compiler"


def test_an_extension_of_another_torch_is_not_used(build, tmp_path):
    r = run(f"""
import sys, types
old = types.ModuleType("{PKG}._tensors")
old.torch_version, old.bf16_at, old.gradients = "1.0+other", None, None
sys.modules[old.__name__] = old
import torch, {PKG} as lm
x = torch.zeros(8, 64, dtype=torch.bfloat16)
try:
    lm.lmoe_gated_ffn(x, x, x, x)
except ImportError as e:
    assert "another torch" in str(e) and "__graft_entry__" in str(e), e
else:
    raise AssertionError("called")
""", ROOT)
    assert r.returncode == 0, r.stderr
