"""What the build makes where torch is missing or has changed (the compilers
are stood in for; nothing is compiled here)."""
from __future__ import annotations

import os
import sys

import pytest

from async_barrier_pipelined_gb300 import build as b


@pytest.fixture
def made(monkeypatch, tmp_path):
    """Empty _lib, and a list of what was built in it."""
    log = []
    lib = str(tmp_path)
    monkeypatch.setattr(b, "LIB_DIR", lib)
    monkeypatch.setattr(b, "LIB_PATH", os.path.join(lib, "lib.so"))
    monkeypatch.setattr(b, "CALLS_PATH", os.path.join(lib, "calls.so"))
    monkeypatch.setattr(b, "CALLS_STAMP", os.path.join(lib, "calls.for"), raising=False)

    def write(path):
        with open(path, "w") as f:
            f.write("built")

    def library(force, verbose):
        log.append("library")
        write(b.LIB_PATH)
        return b.LIB_PATH

    class Compiler:
        def __init__(self, cmd):
            log.append("calls")
            write(cmd[-1])

        def wait(self):
            return 0

        def poll(self):
            return 0

    monkeypatch.setattr(b, "_build_library", library)
    monkeypatch.setattr(b, "_link_calls", lambda obj, out: write(out))
    monkeypatch.setattr(b.subprocess, "Popen", Compiler)
    return log


def test_the_library_is_built_without_torch(made, monkeypatch):
    for name in [m for m in sys.modules if m == "torch" or m.startswith("torch.")]:
        monkeypatch.delitem(sys.modules, name)
    monkeypatch.setitem(sys.modules, "torch", None)     # `import torch` fails
    assert b.build() == b.LIB_PATH and os.path.exists(b.LIB_PATH)
    assert made == ["library"] and not os.path.exists(b.CALLS_PATH)


def test_the_calls_are_built_once_per_torch(made, monkeypatch):
    pytest.importorskip("torch")
    monkeypatch.setattr(b, "_calls_cmd", lambda obj: ["compile", obj])
    for _ in range(2):
        b.build()
    assert made == ["calls", "library", "library"]
    monkeypatch.setattr(b.importlib.metadata, "version", lambda name: "99.0")
    for _ in range(2):
        b.build()
    assert made[3:] == ["calls", "library", "library"]


def test_what_is_there_but_has_no_stamp_is_built_again(made, monkeypatch):
    pytest.importorskip("torch")
    monkeypatch.setattr(b, "_calls_cmd", lambda obj: ["compile", obj])
    b.build()
    os.remove(b.CALLS_STAMP)
    b.build()
    assert made.count("calls") == 2
