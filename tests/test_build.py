"""What the build makes again, and when: the module of the Python bindings fits one torch and may be missing where the
library is there."""
import os
import subprocess
import sys

import pytest
import torch

from speculative_decoding_verify_paged_gb300 import _lib as L
from speculative_decoding_verify_paged_gb300 import build as B


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def test_another_torch_is_not_up_to_date(monkeypatch):
    assert B.up_to_date() and B.calls_fit()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert not B.calls_fit() and not B.up_to_date()


def test_a_missing_module_is_not_up_to_date(monkeypatch, tmp_path):
    monkeypatch.setattr(B, "CALLS", str(tmp_path / "_calls.so"))
    assert not B.calls_fit() and not B.up_to_date()


def test_bindings_build_the_module_that_is_missing(monkeypatch, tmp_path):
    """The library is there and the module is not: the first call of a binding builds it and goes on (here until it
    meets its argument)."""
    made = []
    monkeypatch.setattr(B, "CALLS_FOR", str(tmp_path / "calls_for"))
    monkeypatch.setattr(B, "build_calls", lambda: made.append(1))
    monkeypatch.setattr(L, "_calls", None)
    module = L._bound()
    assert made == [1] and module is L._calls
    with pytest.raises(TypeError):
        module.qk_norm_rope(None, torch.zeros(1, 1, 8), None, None, None, None, 0)


def test_a_tree_with_the_library_alone(tmp_path):
    """The same in a copy of the package without the built module, in a process of its own."""
    import shutil
    root = os.path.dirname(B.PKG)
    name = os.path.basename(B.PKG)
    shutil.copytree(B.PKG, tmp_path / name, ignore=shutil.ignore_patterns("_calls.so", "_build", "__pycache__"))
    shutil.copytree(os.path.join(root, "include"), tmp_path / "include")
    code = f"from {name} import _lib as L, build as B; L.load(); m = L._bound(); assert B.calls_fit() and m.__file__ == B.CALLS, m.__file__"
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
