"""What the build needs: the library nvcc alone, the binding's native half PyTorch and a host compiler too."""
import sys
import sysconfig

import pytest

from gated_deltanet_mixer_verify_b200 import build as gbuild


def _no_torch(mp):
    mp.setitem(sys.modules, "torch", None)


def _no_python_h(mp):
    mp.setattr(sysconfig, "get_paths", lambda: {"include": "/nowhere"})


def _no_compiler(mp):
    mp.setattr(gbuild, "CXX", "no-such-compiler")


@pytest.mark.parametrize("take_away,name", [(_no_torch, "PyTorch"), (_no_python_h, "Python.h"), (_no_compiler, "no-such-compiler")])
def test_the_library_is_built_without_what_the_binding_needs(monkeypatch, capsys, tmp_path, take_away, name):
    monkeypatch.setattr(gbuild, "needs_build", lambda: False)
    monkeypatch.setattr(gbuild, "BINDING", str(tmp_path / "_binding.so"))       # not there yet
    take_away(monkeypatch)
    assert gbuild.build() == gbuild.LIB
    assert name in capsys.readouterr().err and not (tmp_path / "_binding.so").exists()


def test_the_library_comes_first(monkeypatch):
    done = []
    monkeypatch.setattr(gbuild, "build_library", lambda force, verbose: done.append("library") or gbuild.LIB, raising=False)

    def fail(force=False):
        done.append("binding")
        raise RuntimeError("the compiler's message")

    monkeypatch.setattr(gbuild, "build_binding", fail)
    with pytest.raises(RuntimeError, match="the compiler's message"):
        gbuild.build()
    assert done == ["library", "binding"]


def test_a_binding_built_for_other_versions_is_built_anew_and_never_used(monkeypatch):
    gbuild.build()
    from gated_deltanet_mixer_verify_b200 import gdn
    assert not gbuild.binding_is_stale() and gdn._native().built_for == gbuild.binding_versions()
    monkeypatch.setattr(gbuild, "binding_versions", lambda: "PyTorch 99")
    assert gbuild.binding_is_stale()
    monkeypatch.setattr(gdn, "_native_module", None)
    with pytest.raises(ImportError, match="built for PyTorch .* not for PyTorch 99.*gated_deltanet_mixer_verify_b200.build"):
        gdn._native()
