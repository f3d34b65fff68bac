"""The compiled torch binding is used with the torch that it was built for."""
import pytest

import kimi_delta_attention_30_b200 as kda
from kimi_delta_attention_30_b200 import build


def _module(tmp_path, text):
    f = tmp_path / "_torch_binding.so"
    f.write_bytes(b"\x7fELF..." + text + b"...")
    return str(f)


def test_binding_of_another_torch_is_stale(monkeypatch, tmp_path):
    kda._binding()                                    # built and loaded
    here = build._binding_target()
    assert build.binding_built_for() == here and not build._binding_stale()
    other = here.replace("torch ", "torch 1.", 1)
    for text, says in ((b"", "unknown"), (f"kda binding built for [{other}]".encode(), other)):
        monkeypatch.setattr(build, "BINDING", _module(tmp_path, text))
        assert build.binding_built_for() == says and build._binding_stale()
    monkeypatch.setattr(build, "BINDING", _module(tmp_path, f"kda binding built for [{here}]".encode()))
    assert not build._binding_stale()
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "none.so"))
    assert build._binding_stale()


def test_binding_of_another_torch_is_not_loaded(monkeypatch, tmp_path):
    kda._binding()
    monkeypatch.setattr(kda, "_torch_binding", None)
    monkeypatch.setattr(build, "BINDING", _module(tmp_path, b"kda binding built for [torch 1.0.0 0, cpython-39]"))
    with pytest.raises(RuntimeError, match="built for torch 1.0.0"):
        kda._binding()
