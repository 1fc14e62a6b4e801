"""When the extension module is built again: with its sources, and with the torch and Python that it was built for."""
import os

import pytest
import torch

from mla_latent_kv_12_gb300 import build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A built tree whose compile and link steps only write their files down."""
    for d in ("csrc", "include", "_build"):
        (tmp_path / d).mkdir()
    for f in ("csrc/a.cu", "csrc/binding.cpp", "include/mla.h", "_build/a.o", "libmla.so"):
        (tmp_path / f).write_text("")
    for name, value in dict(PKG=tmp_path, ROOT=tmp_path, CSRC=tmp_path / "csrc", BUILD=tmp_path / "_build",
                            LIB=tmp_path / "libmla.so", NATIVE=tmp_path / "_native.so").items():
        monkeypatch.setattr(B, name, str(value))
    steps = []

    def compile_native(obj, log):
        steps.append("compile")
        with open(obj, "w"):
            return "binding.cpp", 0, ""

    def link_native(obj):
        steps.append("link")
        open(B.NATIVE, "w").close()

    monkeypatch.setattr(B, "_compile_native", compile_native)
    monkeypatch.setattr(B, "_link_native", link_native)
    B.build()
    assert steps == ["compile", "link"]
    steps.clear()
    return steps


def test_nothing_is_built_twice(tree):
    B.build()
    assert tree == []


@pytest.mark.parametrize("change", ["torch", "python", "place"])
def test_another_torch_or_python_builds_it_again(tree, monkeypatch, change):
    if change == "torch":
        monkeypatch.setattr(torch, "__version__", "1.0.0+other")
    elif change == "python":
        soabi = B.sysconfig.get_config_var
        monkeypatch.setattr(B.sysconfig, "get_config_var", lambda name: "other" if name == "SOABI" else soabi(name))
    else:
        monkeypatch.setattr(torch, "__file__", os.path.join(os.sep, "elsewhere", "torch", "__init__.py"))
    B.build()
    assert tree == ["compile", "link"]
    tree.clear()
    B.build()
    assert tree == []


def test_a_link_that_failed_is_made_up_for(tree, monkeypatch):
    def fails(obj):
        raise RuntimeError("link failed")

    os.utime(os.path.join(B.CSRC, "binding.cpp"), (2 ** 31, 2 ** 31))
    link = B._link_native
    monkeypatch.setattr(B, "_link_native", fails)
    with pytest.raises(RuntimeError):
        B.build()
    os.utime(os.path.join(B.CSRC, "binding.cpp"), (1, 1))
    monkeypatch.setattr(B, "_link_native", link)
    tree.clear()
    B.build()
    assert tree[-1:] == ["link"]
