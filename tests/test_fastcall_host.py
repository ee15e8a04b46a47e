"""The binding's fast path is optional: where it cannot be built or loaded, the
library and the Python path serve every call, with a warning. On the CPU."""
import os

import pytest

from decode_attention_static_gb300 import build as da_build


@pytest.fixture()
def elsewhere(tmp_path, monkeypatch):
    """The library built, and the fast path's module to be in an empty folder."""
    library = da_build.build_library()
    path = tmp_path / "_fastcall.so"
    monkeypatch.setattr(da_build, "fastcall_path", lambda: path)
    return library, path


def test_no_toolkit(elsewhere, monkeypatch):
    """With the library up to date, build_library() returns without nvcc."""
    library, path = elsewhere

    def missing():
        raise RuntimeError("nvcc not found")

    monkeypatch.setattr(da_build, "nvcc", missing)
    with pytest.warns(UserWarning, match="fast path was not built: nvcc not found"):
        assert da_build.build_library() == library
    assert not path.exists()


def test_no_compiler(elsewhere, monkeypatch):
    library, path = elsewhere
    monkeypatch.setenv("CXX", str(path.parent / "no-such-compiler"))
    with pytest.warns(UserWarning, match="fast path was not built"):
        assert da_build.build_library() == library
    assert not path.exists()


@pytest.mark.parametrize("how", ["no toolkit", "no compiler", "compile error"])
def test_a_module_that_was_not_rebuilt_is_not_left(elsewhere, monkeypatch, how):
    """A module older than its sources, whose argument lists may not be the
    library's any more, does not outlive a build that fails."""
    library, path = elsewhere
    path.write_bytes(b"an older module")
    os.utime(path, (0, 0))
    if how == "no toolkit":
        monkeypatch.setattr(da_build, "nvcc", lambda: (_ for _ in ()).throw(RuntimeError("nvcc not found")))
    elif how == "no compiler":
        monkeypatch.setenv("CXX", str(path.parent / "no-such-compiler"))
    else:
        monkeypatch.setenv("CXX", "false")
    with pytest.warns(UserWarning, match="fast path was not built"):
        assert da_build.build_library() == library
    assert not path.exists()


def test_a_module_for_another_header_is_not_found(tmp_path, monkeypatch):
    """A module left by another torch, or by sources that moved on, is known by
    the header that its calls were compiled against."""
    now = da_build.fastcall_path()
    text = (da_build.INCLUDE / "decode_attn.h").read_text()
    (tmp_path / "decode_attn.h").write_text(text.replace("int max_pages, int window", "int window, int max_pages"))
    monkeypatch.setattr(da_build, "INCLUDE", tmp_path)
    assert da_build.fastcall_path() != now and da_build.fastcall_path().parent == now.parent
    (tmp_path / "decode_attn.h").write_text(text)
    assert da_build.fastcall_path() == now
