"""The build (CPU only): the C library does not depend on the Python
binding, and a binding made for another torch is not used."""
import os
import shutil

import pytest

from drafter_vocab_top_amd import build as B
from drafter_vocab_top_amd import topk_cols as T


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A build of one source into a folder of its own."""
    for name in ("LIBRARY", "STREAM_LIBRARY", "BINDING_LIBRARY"):
        monkeypatch.setattr(B, name, str(tmp_path / os.path.basename(getattr(B, name))))
    monkeypatch.setattr(B, "OBJDIR", str(tmp_path / "objects"))
    monkeypatch.setattr(B, "SOURCES", [os.path.join(B.CSRC, "topk_round_api.cpp")])
    return tmp_path


def test_the_library_is_built_where_the_binding_does_not_compile(small, monkeypatch):
    bad = small / "bad.cpp"
    bad.write_text("#error no binding\n")
    monkeypatch.setattr(B, "BINDING_SOURCE", str(bad))
    open(B.BINDING_LIBRARY, "w").close()  # of an earlier library
    with pytest.raises(RuntimeError, match="g\\+\\+ failed on the Python binding"):
        B.build()
    assert os.path.exists(B.LIBRARY) and os.path.exists(B.STREAM_LIBRARY)
    assert not os.path.exists(B.BINDING_LIBRARY)


def test_the_library_is_built_without_a_host_compiler(small, monkeypatch):
    monkeypatch.setattr(B, "binding_command", lambda output: [str(small / "no-such-compiler")])
    with pytest.raises(RuntimeError, match="its Python binding is not"):
        B.build()
    assert os.path.exists(B.LIBRARY)


def test_the_library_is_built_without_torch(small, monkeypatch):
    monkeypatch.setattr(B, "built_for", lambda: None)
    assert B.build() == B.LIBRARY and os.path.exists(B.LIBRARY)
    assert not os.path.exists(B.BINDING_LIBRARY) and not B.stale()


def test_a_binding_for_another_torch_is_stale(tmp_path, monkeypatch):
    T._round_binding()  # built
    for name in ("LIBRARY", "BINDING_LIBRARY"):
        copy = str(tmp_path / os.path.basename(getattr(B, name)))
        shutil.copy(getattr(B, name), copy)
        monkeypatch.setattr(B, name, copy)
    assert not B.stale()
    monkeypatch.setattr(B, "built_for", lambda: "torch 0.1, Python 3.10")
    assert B.stale()


def test_a_binding_for_another_torch_is_not_used(monkeypatch):
    assert T._round_binding().built_for == B.built_for()
    monkeypatch.setattr(T, "_round", None)
    monkeypatch.setattr(B, "built_for", lambda: "torch 0.1, Python 3.10")
    with pytest.raises(OSError, match="built for torch"):
        T._round_binding()
