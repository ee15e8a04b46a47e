"""The binding's fast path is optional: where it cannot be built or loaded, the
library and the Python path serve every call, with a warning. On the CPU."""
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
