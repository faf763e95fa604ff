"""When the extension module is built anew: its sources, torch or Python changed (host
logic; the compiler is a stand-in)."""
import os

import pytest
import torch

from exact_attention_117_b200 import build, fa


@pytest.fixture
def runs(tmp_path, monkeypatch):
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_fa_binding.so"))
    made = []

    def run(cmd, check):
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w") as f:
            f.write("x")
        made.append(out)

    monkeypatch.setattr(build.subprocess, "run", run)
    return made


def test_built_once_and_again_for_another_torch(runs, monkeypatch):
    build._build_binding(False, False)
    build._build_binding(False, False)
    assert len(runs) == 1
    monkeypatch.setattr(torch, "__version__", "9.9.9+none")
    build._build_binding(False, False)
    assert len(runs) == 2
    build._build_binding(False, False)
    assert len(runs) == 2
    os.remove(build.BINDING + ".for")
    build._build_binding(False, False)
    assert len(runs) == 3


def test_the_debug_build_builds_it_too(runs, monkeypatch, tmp_path):
    monkeypatch.setattr(build, "DEBUG_LIB", str(tmp_path / "debug.so"))
    build.build(debug=True)
    assert any("_fa_binding" in out for out in runs)


def test_a_module_of_another_torch_is_not_loaded(monkeypatch):
    build.build()
    monkeypatch.setattr(fa, "_native", None)
    monkeypatch.setattr(torch, "__version__", "9.9.9+none")
    with pytest.raises(RuntimeError, match="another torch"):
        fa._load_native()
