"""The tables through which clipping hands tensors to the device, made and
walked on the host (CPU only): no launch of 2^32 threads, every element once."""
import os
import subprocess

import pytest

from lm_head_exact_amd import build as lib_build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.skipif(not os.path.exists(lib_build.HIPCC), reason="needs hipcc")
def test_tables_cover_every_tensor_in_launches_that_fit(tmp_path):
    exe = str(tmp_path / "clip_tables")
    r = subprocess.run([lib_build.HIPCC, "--offload-host-only", "-O1", "-std=c++17", f"-I{lib_build.CSRC}",
                        os.path.join(HERE, "host", "clip_tables.hip"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "every block in place" in r.stdout, r.stdout
