"""Build ``lm_head_exact_amd/libflashsample.so`` for gfx950 with hipcc.

Each translation unit compiles to an object under ``_build/`` (in parallel),
then one shared library is linked in-tree next to this file, so that it
travels with the source tree.  Every call recompiles.
"""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libflashsample.so")
SOURCES = ["fs_configs_dma_a.hip", "fs_configs_dma_b.hip", "fs_configs_dma_ntl.hip", "fs_configs_lds.hip",
           "fs_configs_small.hip", "fs_fused.hip", "fs_api.hip", "fs_unfused.hip",
           "fs_online.hip", "fs_pack.hip", "fs_loss.hip", "fs_clip.hip",
           "fs_logprob.hip", "fs_logprob_grad.hip", "fs_cross_entropy.hip",
           "fs_fp8.hip", "fs_fp8_quantize.hip", "fs_fp8_stream_logits.hip", "fs_fp8_stream_scores.hip",
           "fs_fp8_stream_samples.hip", "fs_fp8_tile_logits.hip", "fs_fp8_tile_scores.hip",
           "fs_fp8_tile_samples.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden",
    "-Wall", "-Wno-unused-result",
    # keep hipcc from forming packed fp32 instructions in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # every multiply and add rounds as written (the score z * (1/T) + g is two
    # roundings); fused multiply-adds only where the source asks for fmaf
    "-ffp-contract=off",
    f"-I{os.path.join(ROOT, 'include')}",
]


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    out = "\n".join(l for l in (r.stdout + r.stderr).splitlines()
                    if "packed-fp32-ops' is not a recognized feature" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{out}")
    if out.strip() and verbose:
        print(out, flush=True)
    return obj


def build(verbose: bool = False) -> str:
    """Compile all sources and link the library; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
