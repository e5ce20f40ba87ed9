"""How the serving operators' compiled binding is built and found (CPU)."""
import os

import pytest
import torch

import tree_speculative_decoding_03_gb300 as tsv
from tree_speculative_decoding_03_gb300 import builder


@pytest.fixture
def fresh(monkeypatch):
    monkeypatch.setattr(tsv, "_marshal_module", None)


def test_its_name_holds_what_it_was_built_against():
    import sysconfig
    path = builder.marshal_path()
    assert sysconfig.get_config_var("SOABI") in path and torch.__version__.split("+")[0] in path
    tsv.build()
    assert os.path.exists(path) and tsv._marshal() is not None


def test_one_built_against_another_torch_is_not_loaded(fresh, monkeypatch):
    tsv.build()
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    with pytest.raises(RuntimeError, match="not built.*run build"):
        tsv._marshal()


@pytest.mark.parametrize("without", ["Python.h", "torch/csrc/autograd/python_variable.h"])
def test_the_library_is_built_without_torchs_or_pythons_headers(fresh, monkeypatch, tmp_path, without):
    # include folders that lack the one header, and no binding built yet
    dirs = [d for d in builder._marshal_includes() if not os.path.exists(os.path.join(d, without))]
    monkeypatch.setattr(builder, "_marshal_includes", lambda: dirs)
    monkeypatch.setattr(builder, "marshal_path", lambda: str(tmp_path / "_marshal.so"))
    with pytest.warns(RuntimeWarning, match=without):
        assert os.path.exists(tsv.build())
    assert tsv.load().tsv_last_error() is not None and os.listdir(tmp_path) == []
    one = torch.zeros(1)
    with pytest.raises(RuntimeError, match=f"building it needs {without}"):  # loudly, and only these calls
        tsv.decode_attn(one, one, one, one, one, one, 1.0)


def test_the_library_is_built_without_torch(fresh, monkeypatch, tmp_path):
    def missing():
        raise ImportError("no torch")

    monkeypatch.setattr(builder, "_marshal_includes", missing)
    with pytest.warns(RuntimeWarning, match="torch not found"):
        assert os.path.exists(tsv.build())


def test_a_binding_that_does_not_compile_is_an_error(fresh, monkeypatch, tmp_path):
    bad = tmp_path / "marshal.cpp"
    bad.write_text("int f( {")
    monkeypatch.setattr(builder, "MARSHAL_SRC", str(bad))
    monkeypatch.setattr(builder, "marshal_path", lambda: str(tmp_path / "_marshal.so"))
    with pytest.raises(RuntimeError, match="compiling marshal.cpp failed"):
        tsv.build()
