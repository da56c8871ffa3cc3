"""What build_lib builds, and when: the C library without PyTorch, the binding of the paged calls again for another one.
Compilers are replaced by a record of their calls."""
import os

import pytest

from attention_fa_fwd_03_gb300 import build_lib


@pytest.fixture
def compilers(monkeypatch, tmp_path):
    """Build into an empty folder; -> the outputs that were asked for, in order."""
    for name, at in (("LIB", "lib.so"), ("BINDING", "_paged.so"), ("BUILD", "b"), ("BINDING_FOR", "b/paged_binding.pytorch")):
        monkeypatch.setattr(build_lib, name, os.path.join(tmp_path, at))
    made = []

    def compile_(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        made.append((os.path.basename(cmd[0]), os.path.basename(out).split(".tmp")[0]))
        with open(out, "w"):
            pass

        class Done:
            returncode = 0

            def wait(self):
                return 0
        return Done()

    monkeypatch.setattr(build_lib.subprocess, "Popen", compile_)
    monkeypatch.setattr(build_lib.subprocess, "run", compile_)
    return made


def test_without_pytorch_the_library_is_built(compilers, monkeypatch):
    monkeypatch.setattr(build_lib, "_pytorch", lambda: None)

    def flags():
        raise ImportError("no PyTorch")

    monkeypatch.setattr(build_lib, "_binding_flags", flags)
    assert not build_lib.up_to_date()
    assert build_lib.build() == build_lib.LIB
    assert {c for c, _ in compilers} == {"nvcc"} and os.path.exists(build_lib.LIB)
    assert not os.path.exists(build_lib.BINDING)
    assert build_lib.up_to_date()
    compilers.clear()
    build_lib.build()
    assert compilers == []


def test_pytorch_missing_altogether(monkeypatch):
    import importlib.util
    monkeypatch.setattr(importlib.util, "find_spec", lambda name: None)
    assert build_lib._pytorch() is None


def test_the_binding_follows_pytorch(compilers, monkeypatch):
    monkeypatch.setattr(build_lib, "_pytorch", lambda: "1.0 /a cpython-312")
    build_lib.build()
    assert ("g++", "_paged.so") in compilers and ("nvcc", "lib.so") in compilers
    assert build_lib.up_to_date()
    compilers.clear()
    build_lib.build()
    assert compilers == []
    # another PyTorch: its binding alone is built again
    monkeypatch.setattr(build_lib, "_pytorch", lambda: "2.0 /a cpython-312")
    assert not build_lib.up_to_date()
    build_lib.build()
    assert compilers == [("g++", "paged_binding.o"), ("g++", "_paged.so")]
    assert build_lib.up_to_date()


def test_flags_that_fail_start_no_compiler(compilers, monkeypatch):
    def flags():
        raise ImportError("PyTorch does not import")

    monkeypatch.setattr(build_lib, "_binding_flags", flags)
    with pytest.raises(ImportError):
        build_lib.build()
    assert compilers == []
