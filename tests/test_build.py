"""What a build needs: the library only the HIP compiler, the Python module torch as well."""
import os
import subprocess
import sys

import pytest

from weight_only_bit_moe_amd import build as B


@pytest.fixture
def dry_build(monkeypatch, tmp_path):
    """build() with nothing to compile and a link that writes an empty file."""
    monkeypatch.setattr(B, "SOURCES", [])
    monkeypatch.setattr(B, "PKG", str(tmp_path))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(B, "MODULE", str(tmp_path / "module.so"))
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, b"", b"")
    monkeypatch.setattr(B.subprocess, "run", run)
    return ran


def test_build_without_torch_builds_the_library(dry_build, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert B.build() == B.LIB and os.path.exists(B.LIB)
    assert not os.path.exists(B.MODULE)
    assert "torch" in capsys.readouterr().err


def test_build_without_gxx_uses_hipccs_compiler(dry_build, monkeypatch):
    which = B.shutil.which
    monkeypatch.setattr(B.shutil, "which", lambda n: None if n == "g++" else which(n))
    B.build()
    assert os.path.exists(B.MODULE)
    assert os.path.basename(dry_build[-1][0]) == "clang++" and os.path.exists(dry_build[-1][0])
