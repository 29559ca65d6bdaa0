"""Code-generation checks of the cross entropy's and the 8-bit head's kernels (host
only: compiles their translation units to gfx950 assembly and reads it): the tile
loops' counted waits cover what their barriers publish, and registers hold
everything."""
import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

import test_codegen_tiles as tiles

UNITS = ("fs_cross_entropy.hip", "fs_fp8_tile_scores.hip", "fs_fp8_tile_samples.hip", "fs_fp8_tile_logits.hip",
         "fs_fp8_stream_scores.hip", "fs_fp8_stream_samples.hip")

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None and
                                not os.path.exists("/opt/rocm/bin/hipcc"), reason="needs hipcc")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Assembly lines and scratch bytes of every kernel, by demangled name."""
    outdir = str(tmp_path_factory.mktemp("asm"))
    with ThreadPoolExecutor(len(UNITS)) as ex:
        texts = list(ex.map(lambda u: tiles._assemble(u, outdir), UNITS))
    found = {}
    for s in texts:
        names = re.findall(r"^\s*\.amdhsa_kernel (\S+)", s, re.M)
        plain = subprocess.run(["c++filt"], input="\n".join(names), capture_output=True,
                               text=True).stdout.splitlines()
        for n, d in zip(names, plain):
            start = s.index("\n" + n + ":")
            body = s[start:s.index(".Lfunc_end", start)].splitlines()
            scratch = int(re.search(r"private_segment_fixed_size (\d+)",
                                    s[s.index(".amdhsa_kernel " + n):]).group(1))
            found[d] = (body, scratch)
    return found


def test_cross_entropy_waits(kernels):
    some = {n: k for n, k in kernels.items() if "xent_logits_kernel" in n}
    assert len(some) == 18, sorted(some)
    tiles.test_waits_cover_what_the_barriers_publish(some)


def test_8_bit_tile_waits(kernels, monkeypatch):
    def shape(name):
        wa, wb, mr, nt, s = (int(x) for x in re.search(
            r"Fp8Tile<(\d+), (\d+), (\d+), (\d+), (\d+)>", name).groups())
        return s, (wa * mr + wb * nt) * 32 * 128 // (wa * wb * 1024)
    # from the first staging load on: a barrier before it publishes the scales
    some = {}
    for n, (lines, scratch) in kernels.items():
        if "fp8_tile_kernel" in n:
            first = next(i for i, x in enumerate(lines) if re.match(r"\s*buffer_load\S* .*\blds\b", x))
            some[n] = (lines[first:], scratch)
    assert len(some) == 25, sorted(some)  # (scores by exact products too)
    monkeypatch.setattr(tiles, "_shape", shape)
    tiles.test_waits_cover_what_the_barriers_publish(some)


def test_registers_hold_everything(kernels):
    assert len([n for n in kernels if "fp8_stream_kernel" in n]) == 40
    for name, (_, scratch) in kernels.items():
        assert scratch == 0, f"{name}: {scratch} bytes of scratch"
