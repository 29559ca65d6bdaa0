"""Which tile the rule takes for the logits of the GPU tests' shapes (CPU only:
the rule is compiled for the host), so that a change of the rule cannot leave a
tile without a test."""
import os
import subprocess

import pytest

import test_gpu_logprob_tiles as grad_tests
import test_gpu_token_logprobs as forward_tests
from lm_head_exact_amd import build as lib_build

HERE = os.path.dirname(os.path.abspath(__file__))
TILES = {(256, 64), (256, 128), (256, 256), (64, 64), (64, 128), (128, 128)}


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    if not os.path.exists(lib_build.HIPCC):
        pytest.skip("needs hipcc")
    exe = str(tmp_path_factory.mktemp("rule") / "tile_rule")
    r = subprocess.run([lib_build.HIPCC, "--offload-host-only", "-O1", "-std=c++17", f"-I{lib_build.CSRC}",
                        os.path.join(HERE, "host", "tile_rule.hip"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]

    def tiles(shapes, some):
        out = subprocess.run([exe], input="".join(f"{B} {V} {some}\n" for B, V in shapes),
                             capture_output=True, text=True, check=True).stdout
        return [tuple(int(x) for x in line.split()) for line in out.splitlines()]
    return tiles


def test_gradient_cases_take_the_tiles_that_they_name(rule):
    cases = grad_tests.CASES
    assert rule([(B, V) for B, _, V, _ in cases], 1) == [t for *_, t in cases]
    assert {t for *_, t in cases} == TILES


def test_forward_cases_take_the_tiles_that_they_name(rule):
    cases = grad_tests.FORWARD
    assert rule([(B, V) for B, _, V, _ in cases], 0) == [t for *_, t in cases]
    assert all(D % 32 == 0 for _, D, _, _ in cases)   # (both layouts of W)
    assert {t for B, _, _, t in cases if B > t[1]} == TILES
    # those of one tile's tokens that read W in fragment order past the caches
    assert {t for B, _, _, t in cases if B <= t[1]} >= {(64, 64), (64, 128), (256, 64), (256, 128)}


def test_older_forward_cases_take_every_tile(rule):
    (mark,) = [m for m in forward_tests.test_every_tile.pytestmark if m.name == "parametrize"]
    assert set(rule([(B, V) for B, _, V in mark.args[1]], 0)) == TILES
