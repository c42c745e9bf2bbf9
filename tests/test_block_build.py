"""The build of the block operators' binding beside the library."""
import ctypes
import shutil
import sysconfig

import pytest
import torch

from gated_deltanet_linear_chunk_gb300 import build


def test_binding_is_named_by_what_it_was_compiled_for(monkeypatch):
    """An interpreter or PyTorch of another version has no binding yet, rather
    than one compiled against other headers."""
    path = build.binding_path()
    assert sysconfig.get_config_var("SOABI") in path and torch.__version__ in path
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    assert build.binding_path() != path
    monkeypatch.undo()
    real = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var",
                        lambda name: "cpython-00-other" if name == "SOABI" else real(name))
    assert build.binding_path() != path


@pytest.mark.skipif(shutil.which("nvcc") is None, reason="nvcc not installed")
def test_library_is_linked_without_a_binding(monkeypatch, tmp_path):
    """C users need nvcc alone: where the binding cannot be compiled the library
    is there all the same, and the build says what failed."""
    src = tmp_path / "empty.cu"
    src.write_text('extern "C" __attribute__((visibility("default"))) int gdn_empty() { return 1; }\n')
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "out"))
    monkeypatch.setattr(build, "_sources", lambda: [str(src)])

    def none(out):
        raise FileNotFoundError("Python.h")
    monkeypatch.setattr(build, "_binding_command", none)
    with pytest.raises(FileNotFoundError, match="Python.h"):
        build.build(debug=False)
    assert ctypes.CDLL(build.library_path(False)).gdn_empty() == 1
    monkeypatch.setattr(build, "_binding_command", lambda out: ["false"])
    with pytest.raises(RuntimeError, match="block_binding"):  # the library is up to date
        build.build(debug=False)
