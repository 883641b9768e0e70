"""The binding module is compiled again for another torch: it links to that torch's C++ interface."""
import os
import types

import pytest

from audio_driven_talking_b200 import build as fhbuild

torch = pytest.importorskip("torch")


@pytest.fixture
def compiles(monkeypatch, tmp_path):
    """Build folders of their own, and a compiler that only makes the file it is asked for."""
    ran = []

    def run(cmd, **_):
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        ran.append(out)
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(fhbuild, "OBJ", str(tmp_path))
    monkeypatch.setattr(fhbuild, "BIND", str(tmp_path / "bind.so"))
    monkeypatch.setattr(fhbuild, "subprocess", types.SimpleNamespace(run=run))
    return ran


def test_rebuilt_for_another_torch_only(compiles, monkeypatch):
    fhbuild._build_bind(False)
    fhbuild._build_bind(False)
    assert len(compiles) == 1
    monkeypatch.setattr(torch, "__version__", "2.99.0+cu999")
    fhbuild._build_bind(False)
    fhbuild._build_bind(False)
    assert len(compiles) == 2
    fhbuild._build_bind(True)
    os.utime(fhbuild.BIND, (0, 0))          # older than its source
    fhbuild._build_bind(False)
    assert len(compiles) == 4
