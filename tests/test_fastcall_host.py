"""The binding's fast path is optional: where it cannot be built or loaded, the
library and the Python path serve every call, with a warning. On the CPU."""
import importlib.util
import os
import pathlib
import warnings

import pytest
import torch

import decode_attention_static_gb300 as da
from decode_attention_static_gb300 import _binding
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


@pytest.mark.parametrize("content", [None, b"", b"not an ELF file", "another module"],
                         ids=["none", "empty", "garbage", "other"])
def test_a_module_that_does_not_load(elsewhere, monkeypatch, content):
    """The first call of an operator takes the Python path (which here says that
    its tensors are not on a GPU) instead of failing on the module."""
    _, path = elsewhere
    if content == "another module":
        content = pathlib.Path(_another_module()).read_bytes()
    if content is not None:
        path.write_bytes(content)
    monkeypatch.setattr(_binding, "_fast", None)
    q, cache = torch.zeros(1, 2, 64, dtype=torch.float16), torch.zeros(1, 1, 16, 64, dtype=torch.float16)
    n = torch.ones(1, dtype=torch.int32)
    with warnings.catch_warnings(record=True) as said:
        warnings.simplefilter("always")
        with pytest.raises(ValueError, match="CUDA"):
            da.decode_attn_window_fwd(q, cache, cache, n, 4)
    assert [w for w in said if "fast path does not load" in str(w.message)] or content is None
    assert _binding._fast is False


def _another_module():
    """Some extension module of this Python that is not the fast path's."""
    for name in ("_ctypes", "_json", "_zoneinfo", "_queue"):
        spec = importlib.util.find_spec(name)
        if spec and spec.origin and spec.origin.endswith(".so"):
            return spec.origin
    pytest.skip("every extension module is built in")


def test_a_tree_that_cannot_be_written(elsewhere, monkeypatch):
    """A module that cannot be rebuilt and not be removed fails no build."""
    library, path = elsewhere
    path.write_bytes(b"an older module")
    os.utime(path, (0, 0))
    monkeypatch.setenv("CXX", "false")

    def refused(self, missing_ok=False):
        raise PermissionError("read-only")

    monkeypatch.setattr(pathlib.Path, "unlink", refused)
    with pytest.warns(UserWarning, match="fast path was not built"):
        assert da_build.build_library() == library


def test_a_warning_that_is_an_error_comes_once(elsewhere, monkeypatch):
    """Where warnings are errors, the first call says that the module does not
    load, and the next one is made."""
    _, path = elsewhere
    path.write_bytes(b"")
    monkeypatch.setattr(_binding, "_fast", None)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(UserWarning, match="does not load"):
            _binding._load_fast()
    assert _binding._fast is False
