"""Which object the native part of the binding is loaded from: only one built for this
interpreter, torch and C ABI, and never beside a library that was replaced meanwhile."""
import os
import shutil

import pytest
import torch

import sm_attn_fwd_b200 as ab
from sm_attn_fwd_b200 import build


@pytest.fixture
def place(tmp_path, monkeypatch):
    """A copy of the built files that the package takes for its own."""
    build.build_ext()
    for name in os.listdir(build.LIBDIR):
        if name.endswith((".so", ".sha")):
            shutil.copy(os.path.join(build.LIBDIR, name), tmp_path)
    monkeypatch.setattr(ab, "_EXT_PATH", str(tmp_path / "attn_torch.so"))
    monkeypatch.setattr(ab, "_LIB_PATH", str(tmp_path / "libattn_b200.so"))
    monkeypatch.setattr(ab, "_ext", None)
    monkeypatch.setattr(build, "EXT", str(tmp_path / "attn_torch.so"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libattn_b200.so"))
    monkeypatch.setattr(build, "LIBDIR", str(tmp_path))
    return tmp_path


def test_the_built_object_is_loaded_and_not_built_again(place):
    before = (place / "attn_torch.so").stat().st_mtime_ns
    assert build.is_current(build.EXT) and build.build_ext() == build.EXT
    assert (place / "attn_torch.so").stat().st_mtime_ns == before
    assert hasattr(ab._native(), "decode_q8")
    assert ab._native() is ab._native()


def other_build(path, part):
    """The object with another digest for its environment (part 0) or its sources (1)."""
    data = path.read_bytes()
    at = data.index(build.EXT_MARK) + len(build.EXT_MARK) + 17 * part
    path.unlink()  # this process may have it mapped
    path.write_bytes(data[:at] + b"0123456789abcdef" + data[at + 16:])


@pytest.mark.parametrize("part", [0, 1])
def test_an_object_of_another_build_is_not_loaded(place, part):
    other_build(place / "attn_torch.so", part)
    with pytest.raises(RuntimeError, match="sm_attn_fwd_b200.build"):
        ab._native()
    assert ab._ext is None


def test_without_the_sources_only_the_environment_counts(place, monkeypatch):
    monkeypatch.setattr(build, "EXT_INPUTS", (str(place / "missing.cpp"),))
    other_build(place / "attn_torch.so", 1)
    assert hasattr(ab._native(), "decode_q8")
    other_build(place / "attn_torch.so", 0)
    assert not build.is_current(build.EXT)


def test_another_torch_makes_it_another_build(place, monkeypatch):
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(RuntimeError, match="torch"):
        ab._native()


def test_a_loaded_library_is_not_replaced(place, monkeypatch):
    """The native part is missing and the library, already loaded, out of date."""
    ab.load_library()
    (place / "attn_torch.so").unlink()
    (place / "libattn_b200.sha").write_text("0123456789abcdef")
    monkeypatch.setattr(build, "build", lambda *a, **k: pytest.fail("the library was rebuilt"))
    with pytest.raises(RuntimeError, match="out of date"):
        ab._native()


def test_a_missing_object_is_built_beside_a_current_library(place, monkeypatch):
    (place / "attn_torch.so").unlink()
    made = []

    def fake(*a, **k):
        made.append(1)
        shutil.copy(os.path.join(os.path.dirname(build.__file__), "_lib", "attn_torch.so"), place)

    monkeypatch.setattr(build, "build_ext", fake)
    assert hasattr(ab._native(), "cache_append") and made == [1]
