"""The compiled torch binding is used with the torch that it was built for."""
import pytest

import kimi_delta_attention_30_b200 as kda
from kimi_delta_attention_30_b200 import build


def test_binding_of_another_torch_is_stale(monkeypatch, tmp_path):
    kda._binding()                                    # built and loaded
    assert build.binding_built_for() == build._binding_target() and not build._binding_stale()
    stamp = tmp_path / "built_for"
    monkeypatch.setattr(build, "BINDING_STAMP", str(stamp))
    assert build.binding_built_for() == "unknown" and build._binding_stale()
    stamp.write_text(build._binding_target().replace("torch ", "torch 1.", 1))
    assert build._binding_stale()
    stamp.write_text(build._binding_target())
    assert not build._binding_stale()


def test_binding_of_another_torch_is_not_loaded(monkeypatch, tmp_path):
    stamp = tmp_path / "built_for"
    stamp.write_text("torch 1.0.0 0, cpython-39")
    kda._binding()
    monkeypatch.setattr(kda, "_torch_binding", None)
    monkeypatch.setattr(build, "BINDING_STAMP", str(stamp))
    with pytest.raises(RuntimeError, match="built for torch 1.0.0"):
        kda._binding()
