"""The package without its C++ binding, and when the build makes the binding anew."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

import pytest
import torch

import looped_transformer_decode_b200 as lla
from looped_transformer_decode_b200 import build as B

PKG = os.path.dirname(os.path.abspath(lla.__file__))


def without_binding(tmp_path, code, garbage=False):
    """Runs code on a copy of the package whose binding is missing, or not a library."""
    to = tmp_path / "looped_transformer_decode_b200"
    to.mkdir()
    for name in os.listdir(PKG):
        if name.endswith((".py", "liblla.so")):
            shutil.copy(os.path.join(PKG, name), to / name)
    if garbage:
        (to / "_binding.so").write_bytes(b"not a library")
    return subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True,
                          timeout=600, env={**os.environ, "PYTHONPATH": str(tmp_path)})


CODE = """
import torch, looped_transformer_decode_b200 as lla
assert lla.__file__.startswith({where!r}), lla.__file__
cfg = lla.Cfg(4, 2, 64, 16, 32)
assert lla.ratio(cfg) == lla.Fraction(32, 3)
assert lla.decode_launches(cfg, 2, 100) > 0 and lla.q8_decode_launches(cfg, 1, 64) == 1
one = torch.zeros(1, dtype=torch.int32)
try:
    lla.page_map(16, one, one, one.view(1, 1), one, one, 4)
except ImportError as e:
    assert "page_map" in str(e) and "build" in str(e), e
else:
    raise SystemExit("no error")
"""


def test_package_imports_without_the_binding(tmp_path):
    for garbage in (False, True):
        where = tmp_path / str(garbage)
        where.mkdir()
        r = without_binding(where, CODE.format(where=str(where)), garbage)
        assert r.returncode == 0, r.stdout + r.stderr


@pytest.fixture
def builds(tmp_path, monkeypatch):
    """The build with outputs of its own and a compiler that only counts: a list of its commands."""
    ran = []
    monkeypatch.setattr(B, "BUILD", str(tmp_path))
    monkeypatch.setattr(B, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(B, "BINDING_FOR", str(tmp_path / "binding.txt"))

    def run(cmd, check):
        ran.append(cmd)
        (tmp_path / "_binding.so").write_bytes(b"")

    monkeypatch.setattr(B.subprocess, "run", run)
    return ran


def test_binding_is_built_anew_for_another_torch_or_python(builds, monkeypatch):
    B.build_binding()
    B.build_binding()
    assert len(builds) == 1
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    B.build_binding()
    B.build_binding()
    assert len(builds) == 2
    monkeypatch.setattr(B.sys, "version", "2.7")
    B.build_binding()
    B.build_binding()
    assert len(builds) == 3
    os.remove(B.BINDING_FOR)                     # not known what it was built for
    B.build_binding()
    assert len(builds) == 4
    B.build_binding(force=True)
    assert len(builds) == 5


def test_a_failed_build_leaves_no_mark(builds, monkeypatch):
    B.build_binding()

    def fail(cmd, check):
        raise subprocess.CalledProcessError(1, cmd)

    monkeypatch.setattr(B.subprocess, "run", fail)
    with pytest.raises(subprocess.CalledProcessError):
        B.build_binding(force=True)
    assert not os.path.exists(B.BINDING_FOR)
