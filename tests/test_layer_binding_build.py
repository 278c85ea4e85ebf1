"""Without its direct binding (csrc/binding.cpp) the package still builds and
every call takes the general path; that it does so is said."""
import os

import pytest

from hybrid_linear_attention_deltanet_gb300 import _build


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
