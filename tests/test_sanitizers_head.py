"""The host paths of the cross entropy and of the 8-bit head (argument checks, size
arithmetic, tile rules, the fault-injection hook) under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): the translation units are compiled with
the sanitizers on the host side only (-Xarch_host), linked with the kernels'
objects of the regular build, and driven by tests/sanitize/head_driver.c; nothing is
launched."""
import os
import subprocess

import pytest

from lm_head_exact_amd import build as lib_build
from test_sanitizers import CLANG, HERE, HIPCC, HOST_TUS, ROOT, _env, _run

UNITS = HOST_TUS + ["fs_logprob", "fs_logprob_grad", "fs_cross_entropy", "fs_fp8", "fs_fp8_quantize"]


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="needs ROCm hipcc")
def test_head_host_paths_under_asan_and_ubsan(tmp_path):
    kernels = [os.path.join(ROOT, "_build", os.path.splitext(src)[0] + ".o")
               for src in lib_build.SOURCES if src.startswith(("fs_configs_", "fs_fp8_stream_", "fs_fp8_tile_"))]
    if not kernels or not all(os.path.exists(k) for k in kernels):
        pytest.skip("kernels' objects missing: run the library build first")
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-fvisibility=hidden",
             "-w", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer",
             "-ffp-contract=off", f"-I{os.path.join(ROOT, 'include')}"]
    procs, objs = [], []
    for tu in UNITS:
        obj = str(tmp_path / f"{tu}.o")
        objs.append(obj)
        procs.append(subprocess.Popen(
            [HIPCC, *flags, "-c", os.path.join(ROOT, "lm_head_exact_amd", "csrc", f"{tu}.hip"),
             "-o", obj], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    for tu, p in zip(UNITS, procs):
        out, _ = p.communicate(timeout=600)
        assert p.returncode == 0, f"{tu}: {out}"
    lib = str(tmp_path / "libflashsample_san.so")
    _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-Xarch_host", "-fsanitize=address",
          "-Xarch_host", "-fsanitize=undefined", *objs, *kernels, "-o", lib])
    exe = str(tmp_path / "head_san")
    _run([CLANG, "-std=c11", "-O1", "-g", "-fsanitize=address,undefined",
          "-fno-sanitize-recover=all", "-fno-omit-frame-pointer",
          f"-I{os.path.join(ROOT, 'include')}", os.path.join(HERE, "head_driver.c"), "-o", exe,
          f"-L{tmp_path}", "-lflashsample_san", f"-Wl,-rpath,{tmp_path}", "-lm"])
    r = _run([exe], env=_env(ASAN_OPTIONS="detect_leaks=1", UBSAN_OPTIONS="halt_on_error=1"))
    assert "all head host paths ran clean" in r.stdout
