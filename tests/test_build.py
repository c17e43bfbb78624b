"""What build() makes and when, with the compilers replaced by fakes."""
import os

import pytest

from q8_quantized_matmul_gb300 import build as b


@pytest.fixture
def fake(monkeypatch, tmp_path):
    """build() into a folder of its own; -> the list of what was compiled."""
    made = []

    def out(name, path):
        made.append(name)
        with open(path, "w") as f:
            f.write(name)

    monkeypatch.setattr(b, "LIB", str(tmp_path / "libq8.so"))
    monkeypatch.setattr(b, "TORCH_EXT", str(tmp_path / "_q8torch.so"))
    monkeypatch.setattr(b, "OBJ", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "_compile", lambda src, extra: src)
    monkeypatch.setattr(b, "_link", lambda objs: out("lib", b.LIB))
    monkeypatch.setattr(b, "_compile_torch", lambda: out("ext", b.TORCH_EXT))
    monkeypatch.setattr(b, "torch_version", lambda: "2.9.1")
    return made


def test_the_library_is_built_without_torch(fake, monkeypatch):
    monkeypatch.setattr(b, "torch_version", lambda: None)
    monkeypatch.setattr(b, "_compile_torch", lambda: pytest.fail("torch is not there"))
    assert b.stale() and b.build() == b.LIB
    assert fake == ["lib"] and not b.stale()
    b.build()
    b.build(force=True)
    assert fake == ["lib", "lib"]
    # torch comes later: its module alone is missing
    monkeypatch.setattr(b, "torch_version", lambda: "2.9.1")
    monkeypatch.setattr(b, "_compile_torch", lambda: (fake.append("ext"), open(b.TORCH_EXT, "w").close()))
    assert b.stale()
    b.build()
    assert fake == ["lib", "lib", "ext"] and not b.stale()


def test_an_error_of_the_helpers_leaves_the_library(fake, monkeypatch):
    def broken():
        raise RuntimeError("g++ failed")
    monkeypatch.setattr(b, "_compile_torch", broken)
    with pytest.raises(RuntimeError, match="g.. failed"):
        b.build()
    assert fake == ["lib"] and os.path.exists(b.LIB) and b.stale()


def test_another_torch_makes_the_helpers_stale(fake, monkeypatch):
    b.build()
    assert sorted(fake) == ["ext", "lib"] and not b.stale()
    monkeypatch.setattr(b, "torch_version", lambda: "2.11.0")
    assert b.stale()
    b.build()
    assert fake[2:] == ["ext"] and not b.stale()


def test_versions_are_read_without_importing():
    import torch
    assert b.torch_version() == torch.__version__ or torch.__version__.startswith(b.torch_version())
