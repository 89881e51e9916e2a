"""The build's host side, with the compiler replaced (no nvcc, no GPU)."""
import os
import subprocess
import threading

import pytest

from sparse_attention_video_head_b200 import build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Three sources in a tree of their own; commands go to `calls`, and `-o` names a file that then exists."""
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    for n in ("a", "b", "c"):
        (csrc / f"{n}.cu").write_text("")
    monkeypatch.setattr(B, "CSRC", str(csrc))
    monkeypatch.setattr(B, "INCLUDE", str(csrc))
    monkeypatch.setattr(B, "BUILD_DIR", str(tmp_path / "build"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "lib.so"))
    calls = []

    def run(cmd):
        calls.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
    monkeypatch.setattr(B.subprocess, "check_call", run)
    return csrc, calls, run


def test_stale_sources_are_compiled_side_by_side(tree, monkeypatch):
    csrc, calls, run = tree
    monkeypatch.setattr(os, "cpu_count", lambda: 4)
    together = threading.Barrier(3)

    def compile_or_link(cmd):
        if "-c" in cmd:
            together.wait(timeout=30)  # broken unless all three compile at once
        run(cmd)
    monkeypatch.setattr(B.subprocess, "check_call", compile_or_link)
    assert B.build() == B.LIB
    assert len(calls) == 4 and "-shared" in calls[-1]
    assert [os.path.basename(o) for o in calls[-1][-3:]] == ["a.o", "b.o", "c.o"]


def test_only_what_changed_is_compiled(tree):
    csrc, calls, _ = tree
    B.build()
    calls.clear()
    B.build()
    assert not calls
    later = os.path.getmtime(B.LIB) + 5
    os.utime(csrc / "b.cu", (later, later))
    B.build()
    assert [os.path.basename(c[c.index("-o") + 1]) for c in calls][:1] == ["b.o"] and len(calls) <= 2


def test_a_failed_compile_is_raised_and_nothing_is_linked(tree, monkeypatch):
    csrc, calls, run = tree

    def fail_b(cmd):
        if "-c" in cmd and cmd[cmd.index("-c") + 1].endswith("b.cu"):
            raise subprocess.CalledProcessError(1, cmd)
        run(cmd)
    monkeypatch.setattr(B.subprocess, "check_call", fail_b)
    with pytest.raises(subprocess.CalledProcessError):
        B.build()
    assert not os.path.exists(B.LIB) and not any("-shared" in c for c in calls)
