"""The torch module of the 8-bit cache's operators: what its absence breaks, and when it is rebuilt."""
import os
import subprocess

import pytest

import chunked_causal_gqa_gb300 as pkg
from chunked_causal_gqa_gb300 import _binding, build, q8


@pytest.fixture
def apart(tmp_path, monkeypatch):
    """The module's files in a folder of this test; none is there yet and none is loaded."""
    build.build()
    monkeypatch.setattr(build, "EXT", str(tmp_path / "_pfa_torch.so"))
    monkeypatch.setattr(build, "EXT_KEY", str(tmp_path / "_pfa_torch.key"))
    monkeypatch.setattr(q8, "_module", None)
    return tmp_path


def no_compiler(cmd, *args, **kwargs):
    if cmd[0] == "g++":
        raise FileNotFoundError(2, "No such file or directory", "g++")
    return real_run(cmd, *args, **kwargs)


real_run = subprocess.run


def broken_headers(cmd, *args, **kwargs):
    if cmd[0] == "g++":
        return subprocess.CompletedProcess(cmd, 1, "", "fatal error: Python.h: No such file")
    return real_run(cmd, *args, **kwargs)


@pytest.mark.parametrize("run", [no_compiler, broken_headers])
def test_the_library_builds_where_the_module_does_not(apart, monkeypatch, run):
    monkeypatch.setattr(subprocess, "run", run)
    with pytest.warns(UserWarning, match="_pfa_torch.so was not built"):
        assert build.build() == build.LIB
    assert _binding.load(build.LIB).pfa_version() > 0 and pkg.version()[0] == 1
    with pytest.raises(ImportError, match="not found"):
        q8._ext()
    with pytest.raises((OSError, RuntimeError)):
        build.build_extension()


def test_a_module_of_another_torch_is_neither_loaded_nor_kept(apart, monkeypatch):
    env = build.extension_environment()
    for key in ("", "cpython-38 torch 1.0 none cxx11abi 0\nabc\n"):
        (apart / "_pfa_torch.so").write_bytes(b"of another torch")
        (apart / "_pfa_torch.key").write_text(key)
        later = os.path.getmtime(build.EXT_SOURCE) + 1e6         # newer than anything it came from
        os.utime(build.EXT, (later, later))
        with pytest.raises(ImportError, match="build it again"):
            q8._ext()
    monkeypatch.setattr(subprocess, "run", broken_headers)
    with pytest.warns(UserWarning):
        build.build()
    assert not os.path.exists(build.EXT)
    calls = []

    def compiles(cmd, *args, **kwargs):
        calls.append(cmd[0])
        with open(cmd[cmd.index("-o") + 1], "wb") as f:
            f.write(b"module")
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(subprocess, "run", compiles)
    build.build()
    build.build()                                                # once: it is up to date then
    assert calls == ["g++"] and build.built_environment() == env
    build.build_extension(force=True)
    monkeypatch.setattr(build, "extension_environment", lambda: "another")
    build.build()
    assert calls == ["g++"] * 3 and build.built_environment() == "another"
