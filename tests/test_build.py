"""The build on the CPU, its commands recorded instead of run."""

import os
import sys

import pytest

from weight_activation_quantized_amd import _build


@pytest.fixture
def commands(monkeypatch, tmp_path):
    ran = []

    def run(cmd):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(_build, "_run", run)
    monkeypatch.setattr(_build, "LIB_PATH", str(tmp_path / "libmq.so"))
    monkeypatch.setattr(_build, "BINDING_PATH", str(tmp_path / "_mq_torch.so"))
    return ran


def _binding(ran):
    return [c for c in ran if any(a.endswith("torch_binding.cpp") for a in c)]


def test_library_without_torch(commands, monkeypatch, tmp_path, capsys):
    """No torch to import: the C library is built all the same."""
    monkeypatch.setitem(sys.modules, "torch", None)
    monkeypatch.setattr("importlib.util.find_spec", lambda *a, **k: None)
    lib = str(tmp_path / "libmq.so")
    assert _build.build(lib, build_dir=str(tmp_path / "o"), verbose=True) == lib
    assert os.path.exists(lib) and not _binding(commands)
    assert "not built" in capsys.readouterr().out


@pytest.mark.parametrize("abi", [True, False])
def test_binding_takes_torch_s_abi(commands, monkeypatch, tmp_path, abi):
    import torch
    monkeypatch.setattr(torch, "compiled_with_cxx11_abi", lambda: abi)
    _build.build(str(tmp_path / "libmq.so"), build_dir=str(tmp_path / "o"))
    (cmd,) = _binding(commands)
    assert [a for a in cmd if a.startswith("-D_GLIBCXX_USE_CXX11_ABI")] == [f"-D_GLIBCXX_USE_CXX11_ABI={int(abi)}"]
