"""What a build leaves in place when one of its two products cannot be made
(CPU only, the compilers replaced by stand-ins)."""
import os
import sys

import pytest

from nvfp4_block_scaled_07_amd import build as b


@pytest.fixture
def products(tmp_path, monkeypatch):
    """Paths of a library and a marshalling module from an earlier build."""
    lib, binding = tmp_path / "lib.so", tmp_path / "binding.so"
    for f in (lib, binding):
        f.write_text("earlier")
    monkeypatch.setattr(b, "LIB", str(lib))
    monkeypatch.setattr(b, "BINDING", str(binding))
    return lib, binding


def _compilers(monkeypatch, broken=""):
    def run(cmd, verbose):
        if broken and any(broken in str(c) for c in cmd):
            raise RuntimeError(f"{cmd[0]} failed")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("new")
    monkeypatch.setattr(b, "_run", run)


def test_both_are_replaced(products, monkeypatch):
    _compilers(monkeypatch)
    assert b.build() == str(products[0])
    assert [p.read_text() for p in products] == ["new", "new"]


def test_a_failing_marshalling_module_does_not_cost_the_library(products, monkeypatch):
    # and no earlier module stays beside a newer library
    _compilers(monkeypatch, broken="binding.cpp")
    with pytest.raises(RuntimeError, match="failed"):
        b.build()
    assert products[0].read_text() == "new" and not products[1].exists()


def test_without_torch_the_library_is_built(products, monkeypatch, capsys):
    _compilers(monkeypatch)
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch: ImportError
    assert b.build() == str(products[0])
    assert products[0].read_text() == "new" and not products[1].exists()
    assert "torch" in capsys.readouterr().err


def test_a_failing_source_leaves_both_as_they_were(products, monkeypatch):
    _compilers(monkeypatch, broken="norm.hip")
    with pytest.raises(RuntimeError, match="failed"):
        b.build()
    assert [p.read_text() for p in products] == ["earlier", "earlier"]
    assert not [f for f in os.listdir(products[0].parent) if f.endswith(".tmp")]


def test_a_missing_compiler_is_a_build_failure():
    with pytest.raises(RuntimeError, match="no_such_compiler"):
        b._run(["/nonexistent/no_such_compiler", "-o", "x"], False)
    with pytest.raises(RuntimeError, match="failed"):
        b._run([sys.executable, "-c", "import sys; sys.exit('an error')"], False)
