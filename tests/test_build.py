"""The build: libkvo.so for C programs, with or without torch, and the binding against this interpreter's torch (CPU only)."""
import os
import subprocess

import pytest

from sparse_kv_cache_landmark_gb300 import build

PROGRAM = """
#include <stdio.h>
#include "kvo.h"
int main(void) { puts(kvo_last_error(NULL)); return kv_offload_destroy(NULL) == KVO_OK ? 0 : 1; }
"""


def test_a_c_program_linked_by_path_starts_anywhere(tmp_path):
    """No rpath, no LD_LIBRARY_PATH: the program keeps the path that it was linked with."""
    lib = build.build()
    (tmp_path / "main.c").write_text(PROGRAM)
    exe = str(tmp_path / "main")
    subprocess.run(["gcc", "-I", os.path.join(build.ROOT, "include"), str(tmp_path / "main.c"), lib, "-o", exe], check=True)
    env = {k: v for k, v in os.environ.items() if k != "LD_LIBRARY_PATH"}
    r = subprocess.run([exe], cwd="/", env=env, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.fixture
def commands(monkeypatch):
    """What the build would run from here on; nothing is run."""
    build.build()
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    return ran


def test_nothing_is_built_twice(commands):
    build.build()
    assert not commands


def test_another_torch_or_interpreter_builds_the_binding_again(commands, monkeypatch, tmp_path):
    """Whatever the files' times say: an older torch installed later has older files."""
    with open(build.STAMP) as f:
        kept = f.read()
    stamp = tmp_path / "stamp"
    monkeypatch.setattr(build, "STAMP", str(stamp))
    for other in (kept + "x", "", None):
        stamp.unlink(missing_ok=True)
        if other is not None:
            stamp.write_text(other)
            os.utime(stamp, (0, 0))
        del commands[:]
        build.build()
        assert len(commands) == 2 and all(c[0] == "g++" for c in commands), commands      # compile and link
        assert build.BINDING in commands[1] and stamp.read_text() == kept


def test_the_library_needs_no_torch(commands, monkeypatch, capsys):
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    assert build.build() == build.LIB and not commands
    assert "no torch" in capsys.readouterr().err


def test_the_binding_can_be_left_out(commands, monkeypatch):
    monkeypatch.setattr(build, "STAMP", "")          # any look at it would fail
    assert build.build(binding=False) == build.LIB and not commands
