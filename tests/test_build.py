"""When the native parts are rebuilt: _binding.so also for another torch or Python,
whose object layouts it has compiled in."""
import shutil

import pytest
import torch

from sparse_indexed_attention_b200 import build


@pytest.fixture
def built(tmp_path, monkeypatch):
    """A record of the build and what build_library would compile."""
    record, done = tmp_path / "built_for", []
    monkeypatch.setattr(build, "BUILT_FOR", str(record))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "_build_library", lambda verbose: done.append("library"))
    monkeypatch.setattr(build, "_build_binding", lambda: done.append("binding"))
    record.write_text(build.target())
    return record, done


def test_nothing_is_built_twice(built):
    assert not build.is_stale()
    assert build.build_library() == build.LIB and built[1] == []
    build.build_library(force=True)
    assert built[1] == ["library", "binding"]


@pytest.mark.parametrize("change", ["version", "commit", "abi", "python", "no record"])
def test_another_torch_or_python(built, monkeypatch, change):
    record, done = built
    if change == "version":
        monkeypatch.setattr(torch, "__version__", "2.99.0+cu130")
    elif change == "commit":
        monkeypatch.setattr(torch.version, "git_version", "0" * 40)
    elif change == "abi":
        monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    elif change == "python":
        monkeypatch.setattr("sysconfig.get_config_var", lambda name: "cpython-399-x86_64-linux-gnu")
    else:
        record.unlink()
    assert build.binding_is_stale() and build.is_stale() and not build.library_is_stale()
    build.build_library()
    assert done == ["binding"]


def test_a_newer_source(built, monkeypatch):
    monkeypatch.setattr(build, "_inputs", lambda: [__file__])
    monkeypatch.setattr(build.os.path, "getmtime", lambda p: 2.0 if p == __file__ else 1.0)
    build.build_library()
    assert built[1] == ["library", "binding"]


def test_the_record_is_written_after_the_binding(tmp_path, monkeypatch):
    monkeypatch.setattr(build, "BUILT_FOR", str(tmp_path / "built_for"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build, "_binding_command", lambda out: [shutil.which("touch"), out])
    build._build_binding()
    assert (tmp_path / "_binding.so").exists() and (tmp_path / "built_for").read_text() == build.target()
    assert not build.binding_is_stale()
    monkeypatch.setattr(build, "_binding_command", lambda out: [shutil.which("false")])
    with pytest.raises(RuntimeError):
        build._build_binding()
    assert not build.binding_is_stale()               # the one that was there stays
