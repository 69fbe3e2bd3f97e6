"""The build without torch, and for another torch or Python than the module's (on the CPU; nothing is compiled but the
module, once)."""
import importlib.machinery
import os

import pytest

import convolution_backward_b200 as cb
from convolution_backward_b200 import _build

torch = pytest.importorskip("torch")


@pytest.fixture
def kernels_built(monkeypatch):
    """The kernels' libraries as up to date; what else is built is noted."""
    ran = []
    monkeypatch.setattr(_build, "needs_build", lambda: False)
    monkeypatch.setattr(_build, "_build_kernels", lambda: ran.append("kernels"))
    monkeypatch.setattr(_build, "_build_lists", lambda: ran.append("lists"))
    return ran


def test_without_torch_the_libraries_are_built(monkeypatch, kernels_built):
    find = _build.importlib.util.find_spec
    monkeypatch.setattr(_build.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert _build.build() == _build.LIB and kernels_built == []
    assert _build.build(force=True) == _build.LIB and kernels_built == ["kernels"]


def test_the_module_is_this_pythons():
    assert _build.LISTS.endswith(importlib.machinery.EXTENSION_SUFFIXES[0])
    assert os.path.basename(cb._lists().__file__) == os.path.basename(_build.LISTS)
    assert cb._lists().torch_version == torch.__version__.split("+")[0]


def test_another_torch_builds_the_module_again(monkeypatch, tmp_path, kernels_built):
    stamp, module = tmp_path / "torch", tmp_path / "lists.so"
    module.write_text("")
    monkeypatch.setattr(_build, "LISTS", str(module))
    monkeypatch.setattr(_build, "LISTS_FOR", str(stamp))
    _build.build()
    assert kernels_built == ["lists"]            # no word of which torch
    stamp.write_text(_build._torch()[1])
    _build.build()
    assert kernels_built == ["lists"]
    stamp.write_text("1.0")
    _build.build()
    assert kernels_built == ["lists", "lists"]


def test_a_module_of_another_torch_is_refused(monkeypatch):
    monkeypatch.setattr(cb, "_reader", None)
    monkeypatch.setattr(torch, "__version__", "1.0.0+cu128")
    with pytest.raises(cb.DgradUnavailable, match="built against"):
        cb._lists()


def test_the_module_needs_no_cuda_headers(monkeypatch, tmp_path):
    monkeypatch.setattr(_build, "LISTS", str(tmp_path / "lists.so"))
    monkeypatch.setattr(_build, "LISTS_FOR", str(tmp_path / "torch"))
    monkeypatch.setattr(_build, "PKG", str(tmp_path))
    (tmp_path / "_tensor_lists.so").write_text("any Python's")
    commands = []
    run = _build.subprocess.run
    monkeypatch.setattr(_build.subprocess, "run", lambda cmd, **kw: (commands.append(cmd), run(cmd, **kw))[1])
    _build._build_lists()
    assert os.path.exists(tmp_path / "lists.so") and (tmp_path / "torch").read_text() == _build._torch()[1]
    assert not os.path.exists(tmp_path / "_tensor_lists.so")
    assert not any("cuda" in part for part in commands[0] if part.startswith("-I") and "site-packages" not in part)
