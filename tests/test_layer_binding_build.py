"""Without its direct binding (csrc/binding.cpp) the package still builds and
every call takes the general path; that it does so is said."""
import os
import sys

import pytest

import hybrid_linear_attention_deltanet_gb300 as gdn
from hybrid_linear_attention_deltanet_gb300 import _build
from test_abi import lib  # noqa: F401  (fixture)


@pytest.mark.parametrize("compiler", ["/bin/false", "/nonexistent/compiler"])
def test_a_binding_that_does_not_compile_is_left_out(monkeypatch, tmp_path, compiler):
    stale = tmp_path / "_layer_calls.so"
    stale.write_bytes(b"of another build")
    os.utime(stale, (0, 0))
    monkeypatch.setattr(_build, "HERE", str(tmp_path))
    monkeypatch.setenv("CXX", compiler)
    with pytest.warns(RuntimeWarning, match="_layer_calls.so is not built"):
        assert _build.build_binding() is None
    assert list(tmp_path.iterdir()) == []      # nothing that load() would pick up


def test_a_binding_that_does_not_load_is_reported(lib, monkeypatch):  # noqa: F811
    name = gdn.__name__ + "._layer_calls"
    monkeypatch.setitem(sys.modules, name, None)     # its import raises
    monkeypatch.delattr(gdn, "_layer_calls", raising=False)
    monkeypatch.setattr(gdn, "_lib", None)
    monkeypatch.setattr(gdn, "_direct", None)
    with pytest.warns(RuntimeWarning, match="10 to 20 us"):
        gdn.load()
    assert gdn._direct.gated_ffn() is None


def test_a_library_that_lacks_an_entry_point_is_reported(lib, monkeypatch):  # noqa: F811
    calls = pytest.importorskip(gdn.__name__ + "._layer_calls")

    class Lacks:
        @staticmethod
        def bind(path):
            raise ImportError(path + " lacks an entry point")

    monkeypatch.setitem(sys.modules, calls.__name__, Lacks)
    monkeypatch.setattr(gdn, "_layer_calls", Lacks, raising=False)
    monkeypatch.setattr(gdn, "_lib", None)
    monkeypatch.setattr(gdn, "_direct", None)
    with pytest.warns(RuntimeWarning, match="lacks an entry point"):
        gdn.load()
