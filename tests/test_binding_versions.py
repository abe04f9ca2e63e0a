"""The extension module reads torch's and Python's objects by the layout it was
compiled for: one built for others is refused when it is loaded."""
import types

import pytest
import torch

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300.build import build


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


def test_says_what_it_was_built_for():
    b = ops._binding()
    assert torch.__version__.startswith(b.torch_version)
    ops._same_versions(b)


@pytest.mark.parametrize("torch_version,python_version", [("1.0.0", None), (None, 0x0208)])
def test_built_for_another(torch_version, python_version, monkeypatch):
    b = ops._binding()
    other = types.SimpleNamespace(torch_version=torch_version or b.torch_version,
                                  python_version=python_version or b.python_version)
    with pytest.raises(RuntimeError, match="build it again"):
        ops._same_versions(other)
    # the loader asks
    monkeypatch.setattr(ops, "_binding_module", None)
    monkeypatch.setattr(ops.importlib.util, "module_from_spec", lambda spec: other)
    monkeypatch.setattr(ops.importlib.util, "spec_from_file_location",
                        lambda *a: types.SimpleNamespace(loader=types.SimpleNamespace(exec_module=lambda m: None)))
    with pytest.raises(RuntimeError, match="build it again"):
        ops._binding()
