"""The build, as a user of the C library sees it (CPU only)."""
import os
import subprocess

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
