"""The build rules of the extension module that is compiled against torch, without a GPU."""
import os
import shutil

import pytest
import torch

from grouped_gemm_built_gb300 import build, mok


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Copies of the built files, and a stand-in for the compiler."""
    build.build()
    for f in (build.LIB_NAME, build.TORCH_NAME):
        shutil.copy(os.path.join(build.OUT_DIR, f), tmp_path / f)
    if os.path.exists(build.torch_lib_path() + ".tag"):
        shutil.copy(build.torch_lib_path() + ".tag", tmp_path)
    monkeypatch.setattr(build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(mok, "_TORCH_CALLS", None)
    built = []

    def compiler(target):
        built.append(target)
        with open(target + ".tag", "w") as f:
            f.write(build.torch_tag())

    monkeypatch.setattr(build, "_build_torch_calls", compiler)
    return built


def test_an_up_to_date_module_is_not_built_again(tree):
    build.build()
    assert tree == []
    mok.torch_calls()


def test_a_module_of_another_torch_is_built_again(tree, monkeypatch):
    monkeypatch.setattr(torch, "__version__", "2.0.0+other")
    build.build()
    assert tree == [build.torch_lib_path()]
    build.build()
    assert len(tree) == 1


def test_a_module_of_another_torch_is_not_loaded(tree, monkeypatch):
    monkeypatch.setattr(torch, "__version__", "2.0.0+other")
    with pytest.raises(RuntimeError, match="another torch"):
        mok.torch_calls()


def test_the_library_is_built_where_the_module_cannot_be(tmp_path, monkeypatch):
    """Programs that use the C ABI alone need neither torch's headers nor torch."""
    def no_headers(target):
        raise RuntimeError("g++ failed")

    one = [s for s in build.sources() if s.endswith("mok_dropout.cu")]
    monkeypatch.setattr(build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(build, "sources", lambda: one)
    monkeypatch.setattr(build, "_build_torch_calls", no_headers)
    with pytest.raises(RuntimeError, match="failed"):
        build.build()
    assert os.path.exists(tmp_path / build.LIB_NAME)
