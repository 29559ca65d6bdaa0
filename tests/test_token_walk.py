"""The losses' walk over a sequence's tokens, compiled for the host (CPU only):
every token once, none else, for sequences that end anywhere up to 2^31 - 1."""
import os
import subprocess

import pytest

from lm_head_exact_amd import build as lib_build

HOST = os.path.join(os.path.dirname(os.path.abspath(__file__)), "host")


@pytest.mark.skipif(not os.path.exists(lib_build.HIPCC), reason="needs hipcc")
def test_every_token_is_visited_once(tmp_path):
    exe = str(tmp_path / "token_walk")
    r = subprocess.run([lib_build.HIPCC, "--offload-host-only", "-O2", "-std=c++17",
                        f"-I{lib_build.CSRC}", os.path.join(HOST, "token_walk.hip"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "every token once" in r.stdout, r.stdout
