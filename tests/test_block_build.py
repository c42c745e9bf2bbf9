"""The build of the block operators' binding beside the library."""
import sysconfig

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
