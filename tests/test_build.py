"""The build where a part of the toolchain is missing (no GPU): the library and the entry points that need no compiled
binding do not depend on it."""
import os
import subprocess
import sys

import pytest

import block_sparse_streaming_b200 as bss
from block_sparse_streaming_b200 import _build


@pytest.fixture
def other_binding(monkeypatch, tmp_path):
    """A binding of its own, left over from an older source."""
    _build.build()
    source, target = tmp_path / "binding.cpp", tmp_path / "_binding.so"
    target.write_bytes(b"old")
    os.utime(target, (1, 1))
    source.write_text("#error no headers here\n")
    monkeypatch.setattr(_build, "BINDING_SOURCE", str(source))
    monkeypatch.setattr(_build, "BINDING_PATH", str(target))
    return target


def test_library_builds_where_the_binding_does_not_compile(other_binding):
    with pytest.warns(UserWarning, match="(?s)could not be built.*no headers here"):
        assert _build.build() == _build.LIB_PATH
    assert not other_binding.exists()  # not the old one either
    with pytest.raises(RuntimeError, match="no headers here"):
        _build.build_binding()


def test_library_builds_without_a_host_compiler_for_the_binding(other_binding, monkeypatch):
    monkeypatch.setenv("PATH", "/nowhere")
    with pytest.warns(UserWarning, match="could not be built"):
        assert _build.build() == _build.LIB_PATH


def test_entry_points_without_the_binding(tmp_path):
    """Without the binding the paged operators raise when they are first asked for, and nothing else does."""
    code = (f"import sys; sys.path.insert(0, {os.path.dirname(_build.PKG)!r})\n"
            "from block_sparse_streaming_b200 import _build\n"
            f"_build.BINDING_PATH = {str(tmp_path / 'none.so')!r}\n"
            "import block_sparse_streaming_b200 as bss\n"
            "assert bss.launch_count() == 0 and bss.workspace_size(bss.LOZA_OP_DECODE, 2, 0, 4096, 64, 1, 576, 512, "
            "bss.Params(0.07)) >= 0\n"
            "try:\n    bss.loza_rope\nexcept RuntimeError as e:\n    assert 'none.so is missing' in str(e)\n"
            "else:\n    raise SystemExit(1)\n")
    subprocess.run([sys.executable, "-c", code], check=True)
