"""The library and the CPython module beside it are built apart: a host that lacks what the module needs
(torch's or Python's headers, g++) still gets the library, and is told (no GPU needed)."""
import os

import pytest

from gated_delta_rule_81_amd import build


@pytest.mark.parametrize("broken", [RuntimeError("g++ failed for py_cache.cpp"), FileNotFoundError("g++")])
def test_the_library_is_there_without_the_module(tmp_path, monkeypatch, broken):
    lib, module = tmp_path / "libkda.so", tmp_path / "_cache_calls.so"
    module.write_text("of an older library")

    def link(cmd, **_):
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("linked")

    def no_module(verbose):
        raise broken

    monkeypatch.setattr(build, "LIB", str(lib))
    monkeypatch.setattr(build, "CALLS", str(module))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "_compile", lambda src, verbose: src)
    monkeypatch.setattr(build, "_calls", no_module)
    monkeypatch.setattr(build.subprocess, "run", link)
    with pytest.raises(type(broken), match="g\\+\\+"):
        build.build()
    assert os.path.exists(lib) and lib.read_text() == "linked"
    assert not os.path.exists(module)
