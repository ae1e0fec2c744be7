"""When the Python binding is built again, and that one built for another torch is not
used (no GPU)."""
import os
import types

import pytest


@pytest.fixture()
def build():
    from long_context_rope_b200 import build as b
    b.build()
    return b


def test_binding_is_built_again_for_another_torch_or_python(build, monkeypatch, tmp_path):
    import torch
    assert not build._bind_stale()
    now = build.built_for()
    assert str(torch.__version__) in now and "cpython" in now
    built = []
    monkeypatch.setattr(build, "_build_bind", lambda: built.append(1))
    build.build()
    assert not built
    for other in ("torch 2.99.0, cpython-312-x86_64-linux-gnu", now.replace("cpython", "pypy"), ""):
        monkeypatch.setattr(build, "built_for", lambda: other)
        assert build._bind_stale()
        built.clear()
        build.build()
        assert built
    monkeypatch.undo()
    monkeypatch.setattr(build, "BIND_FOR", str(tmp_path / "none"))  # a binding of unknown origin
    assert build._bind_stale()
    assert os.path.exists(build.BIND)


def test_binding_built_for_another_torch_is_refused(build):
    from long_context_rope_b200 import hga
    assert hga._bind.built_for == build.built_for()
    hga._check_built_for(hga._bind)
    for bad in (types.SimpleNamespace(built_for="torch 1.0, cpython-312"), types.SimpleNamespace()):
        with pytest.raises(ImportError, match="build the library again"):
            hga._check_built_for(bad)
