"""The build's list of files: a change to any of them makes the libraries stale."""
import os

import pytest

from sparse_attention_video_tile_b200 import build as B


def test_every_source_and_header_is_listed():
    there = {f for f in os.listdir(B.CSRC) if f.endswith((".cu", ".cpp", ".cuh", ".h"))}
    assert there == set(B.SOURCES + B.HEADERS)
    assert len(B.SOURCES + B.HEADERS) == len(there)


@pytest.mark.parametrize("name", B.SOURCES + B.HEADERS)
def test_a_newer_file_makes_a_library_stale(name, tmp_path, monkeypatch):
    lib = tmp_path / "lib.so"
    lib.write_bytes(b"")
    real = os.path.getmtime
    newer = os.path.join(B.CSRC, name)
    built = max(real(f) for f in [os.path.join(B.CSRC, f) for f in B.SOURCES + B.HEADERS] + [os.path.join(B.INCLUDE, "sta.h")]) + 10
    os.utime(lib, (built, built))
    assert not B._stale(str(lib))
    monkeypatch.setattr(os.path, "getmtime", lambda p: built + 1 if p == newer else real(p))
    assert B._stale(str(lib))
