"""The binding's helper module is rebuilt when torch changes, and not imported
for another torch than its own."""
import os
import subprocess
import sys
import types

import pytest

from cross_layer_top_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture()
def runs(tmp_path, monkeypatch):
    """_build_bind with a compiler that only makes its output file; the list of its command lines."""
    torch_dir = tmp_path / "torch"
    torch_dir.mkdir()
    (torch_dir / "version.py").write_text("__version__ = '9.1.0+x'\ngit_version = 'aa'\n")
    spec = types.SimpleNamespace(submodule_search_locations=[str(torch_dir)])
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: spec)
    monkeypatch.setattr(build, "BIND_LIB", str(tmp_path / "_tensors.so"))
    monkeypatch.setattr(build, "BIND_STAMP", str(tmp_path / "stamp"))
    calls = []

    def run(cmd, **kw):
        calls.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")
    monkeypatch.setattr(build.subprocess, "run", run)
    return calls, torch_dir


def test_rebuilt_for_another_torch(runs):
    calls, torch_dir = runs
    build._build_bind()
    assert len(calls) == 1 and '-DIC_TORCH_VERSION="9.1.0+x"' in calls[0]
    build._build_bind()
    assert len(calls) == 1  # nothing changed
    (torch_dir / "version.py").write_text("__version__ = '9.2.0'\ngit_version = 'bb'\n")
    build._build_bind()
    assert len(calls) == 2 and '-DIC_TORCH_VERSION="9.2.0"' in calls[1]
    (torch_dir / "version.py").write_text("__version__ = '9.2.0'\ngit_version = 'cc'\n")
    build._build_bind()  # the same number, another build
    assert len(calls) == 3
    os.remove(build.BIND_STAMP)  # built before there was one
    build._build_bind()
    build._build_bind()
    assert len(calls) == 4


def test_version_is_torchs_own():
    import torch
    assert build._torch_version(os.path.dirname(torch.__file__)) == torch.__version__


def test_not_imported_for_another_torch():
    build.build()
    code = ("import torch\ntorch.__version__ = '0.1'\n"
            "try:\n    import cross_layer_top_b200.indexcache\n"
            "except ImportError as e:\n    assert 'torch 0.1' not in str(e) and 'this is 0.1' in str(e), e\n"
            "else:\n    raise SystemExit('imported')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
