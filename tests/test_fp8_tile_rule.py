"""Which tile the 8-bit head's rule takes for the GPU tests' shapes (CPU only: the rule
is compiled for the host), so that a change of the rule cannot leave a tile without
a test, and that every call's scales fit in LDS."""
import os
import subprocess

import pytest

import test_gpu_fp8 as gpu_tests
from lm_head_exact_amd import build as lib_build

HERE = os.path.dirname(os.path.abspath(__file__))
TILES = [(256, 64), (256, 128), (256, 256), (128, 128), (64, 64), (64, 64)]


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    if not os.path.exists(lib_build.HIPCC):
        pytest.skip("needs hipcc")
    exe = str(tmp_path_factory.mktemp("rule") / "fp8_tile_rule")
    r = subprocess.run([lib_build.HIPCC, "--offload-host-only", "-O1", "-std=c++17", f"-I{lib_build.CSRC}",
                        os.path.join(HERE, "host", "fp8_tile_rule.hip"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]

    def tiles(shapes):
        out = subprocess.run([exe], input="".join("%d %d %d\n" % s for s in shapes), capture_output=True,
                             text=True, check=True).stdout
        return [tuple(int(x) for x in line.split()) for line in out.splitlines()]
    return tiles


def test_gpu_cases_take_every_tile(rule):
    assert [t[:2] for t in rule(gpu_tests.TILES)] == TILES
    for few in (True, False):
        assert {t[:2] for s, t in zip(gpu_tests.SCORE_TILES, rule(gpu_tests.SCORE_TILES))
                if (s[2] <= 8192) == few} == set(TILES)


def test_scales_fit_beside_the_ring(rule):
    shapes = [(B, D, V) for B in (17, 33, 64, 100, 128, 300, 1000, 4096, 50000)
              for D in (64, 5184, 8192, 12288, 16320, 16384) for V in (1, 2000, 16032, 128256, 151936)]
    assert all(lds <= 160 * 1024 for *_, lds in rule(shapes))
