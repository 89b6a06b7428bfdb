"""What the build and the contexts need (no GPU): the library nvcc alone, the
8-bit calls the extension module, which is built for the installed torch."""
import os

import pytest
import torch

from deepseek_sparse_attention_dsa_gb300 import build as dsa_build
from deepseek_sparse_attention_dsa_gb300 import dsa
from deepseek_sparse_attention_dsa_gb300 import workloads as W


@pytest.fixture(scope="module", autouse=True)
def built():
    dsa_build.build()


@pytest.fixture()
def small(tmp_path, monkeypatch):
    """A build of one translation unit in a folder of its own."""
    monkeypatch.setattr(dsa_build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(dsa_build, "LIB", str(tmp_path / "libdsa_gb300.so"))
    monkeypatch.setattr(dsa_build, "BINDING", str(tmp_path / "_dsa_binding.so"))
    monkeypatch.setattr(dsa_build, "SOURCES", ["selftest.cu"])
    return tmp_path


def test_the_library_is_built_without_torch(small, monkeypatch, capfd):
    def fails():
        raise RuntimeError("no headers")

    monkeypatch.setattr(dsa_build, "_compile_binding", fails)
    (small / "_dsa_binding.so").write_bytes(b"of another torch")
    assert dsa_build.build() == dsa_build.LIB and os.path.exists(dsa_build.LIB)
    assert "no headers" in capfd.readouterr().err
    assert not os.path.exists(dsa_build.BINDING) and not dsa_build.up_to_date() and dsa_build.library_up_to_date()


def test_a_library_that_does_not_compile_is_an_error(small, monkeypatch):
    monkeypatch.setattr(dsa_build, "_compile_binding", lambda: "")
    monkeypatch.setattr(dsa_build, "SOURCES", ["nothing.cu"])
    with pytest.raises(RuntimeError, match="nvcc failed"):
        dsa_build.build()
    assert not os.path.exists(dsa_build.LIB)


def test_the_module_of_another_torch_is_out_of_date(monkeypatch):
    assert dsa_build.up_to_date()
    key = dsa_build._binding_key()
    assert torch.__version__ in key
    monkeypatch.setattr(dsa_build, "_binding_key", lambda: key.replace(torch.__version__, "0.0"))
    assert not dsa_build.up_to_date() and dsa_build.library_up_to_date()


def test_contexts_do_without_the_module(tmp_path, monkeypatch):
    dsa.load()
    monkeypatch.setattr(dsa, "LIB_PATH", str(tmp_path / "libdsa_gb300.so"))
    monkeypatch.setattr(dsa, "_binding", None)
    ctx = dsa.Context(W.DSAShape(**W.DEEPSEEK), device=-1)
    plan = ctx.plan([], 1)
    assert plan.num_rows == 0
    with pytest.raises(RuntimeError, match="_dsa_binding.so is not built"):
        ctx.quantize_rows(torch.zeros(1, 128, dtype=torch.bfloat16))
    monkeypatch.undo()
    with pytest.raises(dsa.DSAError):       # there again: a host-only context is refused by the call itself
        ctx.quantize_rows(torch.zeros(1, 128, dtype=torch.bfloat16))


def test_the_module_of_another_torch_is_not_loaded(monkeypatch):
    dsa.load_binding()
    key = dsa_build._binding_key()
    monkeypatch.setattr(dsa, "_binding", None)
    monkeypatch.setattr(dsa_build, "_binding_key", lambda: key + "0.0")
    with pytest.raises(RuntimeError, match="another torch"):
        dsa.load_binding()
    monkeypatch.undo()
    dsa.load_binding()
