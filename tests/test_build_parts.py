"""What build() compiles, with the compilers replaced by recorders: the C library by nvcc alone, the torch binding
only where there is a torch, and again for another torch."""
import os
import subprocess
import sys
import textwrap

import pytest

from online_softmax_tiling_gb300 import build as b
from tests.test_abi import ROOT


class Tools:
    """Records the compilers' command lines and leaves their output files."""

    def __init__(self, monkeypatch, folder, torch="9.9.9"):
        self.ran = []
        monkeypatch.setattr(b, "LIBRARY", str(folder / "libfa_gb300.so"))
        monkeypatch.setattr(b, "BINDING", str(folder / "_paged_binding.so"))
        monkeypatch.setattr(b, "BINDING_TORCH", str(folder / "_paged_binding.so.torch"))
        monkeypatch.setattr(b, "nvcc", lambda: "nvcc")
        monkeypatch.setattr(b, "_torch_version", lambda: torch)
        monkeypatch.setattr(b.subprocess, "run", self.run)
        monkeypatch.setattr(b.subprocess, "Popen", self.popen)

    def run(self, cmd, check=False):
        self.ran.append(cmd[0])
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass

    def popen(self, cmd):
        self.run(cmd)

        class Done:
            returncode = 0

            def wait(self):
                return 0
        return Done()


def test_library_and_binding(monkeypatch, tmp_path):
    pytest.importorskip("torch")
    t = Tools(monkeypatch, tmp_path)
    assert b.stale()
    b.build()
    assert sorted(t.ran) == ["g++", "g++", "nvcc"] and os.path.exists(b.LIBRARY) and os.path.exists(b.BINDING)
    assert not b.stale()
    b.build()
    assert len(t.ran) == 3
    assert sorted(os.listdir(tmp_path)) == ["_paged_binding.so", "_paged_binding.so.torch", "libfa_gb300.so"]


def test_another_torch_gets_its_own_binding(monkeypatch, tmp_path):
    pytest.importorskip("torch")
    t = Tools(monkeypatch, tmp_path)
    b.build()
    t.ran.clear()
    monkeypatch.setattr(b, "_torch_version", lambda: "9.9.10")
    assert b.stale()
    b.build()
    assert t.ran == ["g++", "g++"] and not b.stale()                 # the library stays
    os.remove(b.BINDING_TORCH)                                       # of an unknown torch
    assert b.stale()


def test_without_a_torch_the_library_alone(monkeypatch, tmp_path):
    t = Tools(monkeypatch, tmp_path, torch=None)
    for force in (False, True):
        t.ran.clear()
        b.build(force=force)
        assert t.ran == ["nvcc"] and not os.path.exists(b.BINDING) and not b.stale()


def test_a_torch_that_cannot_be_imported(tmp_path):
    """In a process whose `import torch` fails, installed or not."""
    code = textwrap.dedent("""
        import os, sys
        sys.modules["torch"] = None
        from online_softmax_tiling_gb300 import build as b
        at, ran = sys.argv[1], []
        b.LIBRARY, b.BINDING, b.BINDING_TORCH = (os.path.join(at, n) for n in ("lib.so", "binding.so", "binding.so.torch"))
        b.nvcc = lambda: "nvcc"
        def run(cmd, check=False):
            ran.append(cmd[0])
            open(cmd[cmd.index("-o") + 1], "w").close()
        b.subprocess.run = run
        for force in (False, True):
            assert b.build(force=force) == b.LIBRARY
        assert ran == ["nvcc", "nvcc"] and os.listdir(at) == ["lib.so"], (ran, os.listdir(at))
        import online_softmax_tiling_gb300 as fa
        assert fa.FA_OK == 0 and "torch" in sys.modules and sys.modules["torch"] is None
    """)
    r = subprocess.run([sys.executable, "-c", code, str(tmp_path)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "not built" in r.stderr or "torch" not in r.stderr
