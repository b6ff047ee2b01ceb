"""The build takes its tools from the ROCm toolchain alone: joining and linking
the objects works without any program on PATH."""
import importlib.util
import os
import subprocess
import types

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "nvfp4_scale_calibration_amd")


def test_objects_are_linked_without_programs_on_path(monkeypatch, tmp_path):
    spec = importlib.util.spec_from_file_location("_lh_build_check", os.path.join(PKG, "_build.py"))
    builder = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(builder)
    if not os.path.exists(builder.HIPCC) or not os.path.exists(os.path.join(PKG, "_build", "lh_api.o")):
        pytest.skip("hipcc or the library's objects are missing (run __graft_entry__.build())")

    class Compiled:                                   # the objects are there: compile nothing
        returncode = 0

        def __init__(self, *args, **kwargs):
            pass

        def communicate(self):
            return "", None

    monkeypatch.setattr(builder, "subprocess", types.SimpleNamespace(
        Popen=Compiled, run=subprocess.run, PIPE=subprocess.PIPE, STDOUT=subprocess.STDOUT))
    monkeypatch.setattr(builder, "LIB", str(tmp_path / "liblh.so"))
    monkeypatch.setenv("PATH", str(tmp_path))
    builder.build()
    data = (tmp_path / "liblh.so").read_bytes()
    assert data[:4] == b"\x7fELF" and b"lh_linear_nvfp4_ragged_grad" in data
