"""Host-only checks of the build: the C library does not depend on the Python module beside it."""
import importlib.metadata
import os

import pytest

from block_sparse_video_vsa_gb300 import build as vbuild


@pytest.fixture
def place(tmp_path, monkeypatch):
    """A build folder of its own, where compiling the library only writes its file."""
    monkeypatch.setattr(vbuild, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(vbuild, "LIB_PATH", str(tmp_path / "libvsa.so"))
    built = []

    def library(verbose):
        built.append("library")
        (tmp_path / "libvsa.so").write_bytes(b"x")

    def front(path):
        built.append("front")
        with open(path, "wb") as f:
            f.write(b"x")

    monkeypatch.setattr(vbuild, "_build_library", library)
    monkeypatch.setattr(vbuild, "_build_front", front)
    return built


def test_library_is_built_without_pytorch(place, monkeypatch):
    def version(name):
        raise importlib.metadata.PackageNotFoundError(name)
    monkeypatch.setattr(importlib.metadata, "version", version)
    assert vbuild.front_path() is None
    assert vbuild.build() == vbuild.LIB_PATH and place == ["library"]
    assert vbuild.up_to_date()


def test_library_is_built_where_the_module_does_not_compile(place, monkeypatch, capsys):
    def front(path):
        raise RuntimeError("no Python.h here")
    vbuild.build()
    path = vbuild.front_path()
    os.utime(path, (1, 1))  # older than its source: stale
    monkeypatch.setattr(vbuild, "_build_front", front)
    assert vbuild.build(force=True) == vbuild.LIB_PATH and place.count("library") == 2
    assert "no Python.h here" in capsys.readouterr().err
    assert not os.path.exists(path)  # a module that does not fit the library is not left to be loaded
    assert not vbuild.up_to_date()


def test_a_stale_module_is_not_up_to_date_and_is_built_again(place):
    vbuild.build()
    assert sorted(place) == ["front", "library"] and vbuild.up_to_date()
    vbuild.build()
    assert len(place) == 2
    os.utime(vbuild.front_path(), (1, 1))
    assert not vbuild.up_to_date()
    vbuild.build()
    assert place.count("front") == 2 and place.count("library") == 1 and vbuild.up_to_date()
