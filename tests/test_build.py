"""What the build makes, with the compilers replaced by one that only writes its output file."""
import os
import subprocess

import pytest

from masked_attention_bound_gb300 import build


@pytest.fixture
def calls(tmp_path, monkeypatch):
    """The commands run so far; g++ fails while the list's `host_fails` is set."""
    class Calls(list):
        host_fails = False

        def count(self, compiler):
            return sum(os.path.basename(c[0]) == compiler for c in self)

    made = Calls()

    def run(cmd, **kw):
        made.append(cmd)
        if made.host_fails and cmd[0] == "g++":
            return subprocess.CompletedProcess(cmd, 1, "", "Python.h: No such file or directory")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(subprocess, "run", run)
    for name, value in (("LIB", "libfm.so"), ("MODULE", "_fmcache.so"), ("BUILD", "objects")):
        monkeypatch.setattr(build, name, str(tmp_path / value))
    return made


def test_the_library_needs_no_host_compiler_for_the_binding(calls):
    """Where the Python module cannot be built, the library is there all the same, and the build
    says what failed, then and the next time."""
    calls.host_fails = True
    with pytest.raises(RuntimeError, match="Python.h"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.MODULE)
    compiled = calls.count("nvcc")
    with pytest.raises(RuntimeError, match="Python.h"):
        build.build()
    assert calls.count("nvcc") == compiled
    calls.host_fails = False
    assert build.build() == build.LIB
    assert os.path.exists(build.MODULE) and calls.count("nvcc") == compiled and build.up_to_date()


def test_the_binding_is_built_again_for_another_torch(calls, monkeypatch):
    import torch
    build.build()
    compiled, host = calls.count("nvcc"), calls.count("g++")
    build.build()
    assert calls.count("g++") == host
    monkeypatch.setattr(torch, "__version__", "99.0")
    assert not build.up_to_date()
    build.build()
    assert calls.count("nvcc") == compiled and calls.count("g++") == 2 * host and build.up_to_date()


def test_force_builds_both(calls):
    build.build()
    compiled, host = calls.count("nvcc"), calls.count("g++")
    build.build(force=True)
    assert calls.count("nvcc") == 2 * compiled and calls.count("g++") == 2 * host
