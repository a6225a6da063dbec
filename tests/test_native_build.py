"""The binding's native part is an addition: without it, or with one for another torch, the package is imported all the
same; the build notices a torch or a Python that is not the one it was built against."""
import importlib.util
import os
import shutil
import subprocess
import sys
import types

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "delta_rule_linear_02_b200")

CALLS = """
import warnings
with warnings.catch_warnings(record=True) as told:
    warnings.simplefilter("always")
    import delta_rule_linear_02_b200 as efla
print("told:", [str(w.message) for w in told if "_efla_native" in str(w.message)])
import torch
assert efla.efla_status_string(efla.EFLA_OK) == "EFLA_OK"
assert efla.efla_scan_workspace_bytes(1, 2, 100, 64, 64) > 0
x = torch.zeros(1, 2, 5, 64)
try:
    efla.efla_scan_fwd(x, x)
except ValueError as e:
    print("refused:", e)
"""


@pytest.fixture
def package(efla, tmp_path):
    """A copy of the package without its native part."""
    to = tmp_path / "delta_rule_linear_02_b200"
    to.mkdir()
    shutil.copy(os.path.join(PKG, "__init__.py"), to)
    os.symlink(os.path.join(PKG, "libefla.so"), to / "libefla.so")

    def run():
        out = subprocess.run([sys.executable, "-c", CALLS], cwd=tmp_path, capture_output=True, text=True, timeout=300)
        assert out.returncode == 0, out.stderr
        assert "refused: x must be on a CUDA device" in out.stdout
        return out.stdout

    return to, run


def test_import_without_the_native_part(package):
    _, run = package
    assert "build.py" in run()


@pytest.mark.parametrize("version", ["0.1", "unknown"])
def test_import_with_one_for_another_torch(package, version):
    to, run = package
    named = f"torch_version = '{version}'\n" if version != "unknown" else ""
    (to / "_efla_native.py").write_text(named + "def bind(*a):\n    raise SystemExit('it was called')\n")
    assert f"built for torch {version}" in run()


def test_import_with_the_one_that_was_built(package):
    to, run = package
    shutil.copy(os.path.join(PKG, "_efla_native.so"), to)
    assert "told: []" in run()


def test_the_build_looks_at_the_torch(efla, tmp_path, monkeypatch):
    spec = importlib.util.spec_from_file_location("efla_build_checked", os.path.join(PKG, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    ran = []
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kw: ran.append(cmd))
    monkeypatch.setattr(build.os, "replace", lambda a, b: None)
    build.build_native()
    assert not ran
    (tmp_path / "version.py").write_text("__version__ = '99.1'\n")
    real = build.importlib.util.find_spec
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name, *a: types.SimpleNamespace(
        submodule_search_locations=[str(tmp_path)]) if name == "torch" else real(name, *a))
    build.build_native()
    assert len(ran) == 1
