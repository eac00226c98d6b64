"""The library builds, imports and checks its calls also where the binding's compiled part cannot be built (CPU only)."""

import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

from io_aware_exact_fa_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The compiled part's files in a folder of their own, with an old one there."""
    build.build()
    for name in ("BINDING", "BINDING_STAMP"):
        monkeypatch.setattr(build, name, str(tmp_path / name))
        (tmp_path / name).write_text("old")
    return tmp_path


def test_without_torch(elsewhere, monkeypatch, capsys):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.BINDING) and "not built" in capsys.readouterr().err


@pytest.mark.parametrize("cxx", ["/no/such/compiler", shutil.which("false") or "false"])
def test_without_a_compiler_that_works(elsewhere, monkeypatch, cxx):
    monkeypatch.setenv("CXX", cxx)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.BINDING)


def test_import_and_refusals_without_the_compiled_part(tmp_path):
    build.build()
    package = tmp_path / "io_aware_exact_fa_gb300"
    package.mkdir()
    for name in os.listdir(os.path.join(ROOT, "io_aware_exact_fa_gb300")):
        if name.endswith(".py"):
            shutil.copy(os.path.join(ROOT, "io_aware_exact_fa_gb300", name), package / name)
    os.symlink(build.LIB, package / "libfa_gb300.so")
    code = """
import torch
from io_aware_exact_fa_gb300 import fa
assert not hasattr(fa._binding, "__file__")
x = torch.zeros(2)
for call in (lambda: fa.append_paged_fp4(x, x, x, x, x, x, x, x, x), lambda: fa.decode_paged_fp4(x, x, x, x, x, x, x),
             lambda: fa.read_paged(x, x, x, x, x, 1), lambda: fa.weigh_paged(x, x, x, x, x, x), lambda: fa.evict_paged(x, x, x, x, x, x, 1)):
    try:
        call()
    except ValueError:
        continue
    raise SystemExit("not refused")
"""
    subprocess.run([sys.executable, "-c", code], cwd=tmp_path, check=True, env={**os.environ, "PYTHONPATH": str(tmp_path)})


def test_the_compiled_part_names_no_type_that_older_torch_lacks():
    with open(os.path.join(build.CSRC, "binding.cpp")) as f:
        assert "kFloat4" not in f.read()
