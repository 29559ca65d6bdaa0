"""Sizes whose launches would hold 2^32 threads or more are refused before
anything is launched; sizes within the stated limits are not (CPU only: with
an injected launch failure nothing runs and the pointers are never touched)."""
import random

import pytest

from lm_head_exact_amd import binding as bd
from test_training_abi import _backward, _logprobs


@pytest.fixture()
def L(monkeypatch):
    monkeypatch.setenv("FS_FAULT_INJECT", "launch")
    return bd.lib()


@pytest.mark.parametrize("fn", ["fs_token_logprobs", "fs_token_logprobs_packed"])
@pytest.mark.parametrize("B,D,V", [
    (1 << 24, 4096, 128256), (5_000_000, 64, 128256), (1 << 24, 96, 151936),
    (33, 5152, 2**31 - 513), (64, 8192, 2**31 - 513), (128, 64, 2**31 - 513), (300, 32, 2**31 - 4096),
])
def test_forward_beyond_a_launch_is_unsupported(L, fn, B, D, V):
    assert _logprobs(L, fn, B=B, D=D, V=V) == bd.FS_ERR_UNSUPPORTED
    assert b"launch grid" in L.fs_last_error()


def test_forward_within_the_stated_limits_is_taken(L):
    r = random.Random(1)
    sizes = [(1, 8, 2**31 - 513), (32, 5120, 2**31 - 513), (33, 8, 2**31 - 4096), (64, 64, 2**31 - 4096),
             (1 << 24, 8, 8192), (1 << 20, 4096, 1 << 17), (257, 64, 2**37 // 257)]
    sizes += [(int(2 ** r.uniform(0, 24)), 64, int(2 ** r.uniform(0, 30.999))) for _ in range(3000)]
    for B, D, V in sizes:
        if V <= 2**31 - 4096 and B * V <= 2**37 or (B <= 16 and V <= 2**31 - 513):
            assert _logprobs(L, B=B, D=D, V=V) == bd.FS_ERR_HIP, (B, V)


@pytest.mark.parametrize("kw", [dict(B=3, D=8, V=1 << 30), dict(B=3, D=8, V=2**31 - 513),
                                dict(B=1 << 22, D=1 << 18, V=100), dict(B=0, D=8, V=1 << 30)])
def test_backward_beyond_a_launch_is_unsupported(L, kw):
    assert _backward(L, **kw) == bd.FS_ERR_UNSUPPORTED
    assert b"launch grid" in L.fs_last_error()


def test_backward_within_the_stated_limits_is_taken(L):
    r = random.Random(2)
    sizes = [(3, 8, (1 << 30) - 256), (1 << 22, 1 << 16, 128256), (1, 1 << 20, 1 << 29), (1 << 22, 8, 1)]
    sizes += [(int(2 ** r.uniform(0, 22)), 8 * int(2 ** r.uniform(0, 17)), int(2 ** r.uniform(0, 29.999)))
              for _ in range(3000)]
    for B, D, V in sizes:
        if B * D <= 2**38:
            assert _backward(L, B=B, D=D, V=V) == bd.FS_ERR_HIP, (B, D, V)
    # without grad_W the vocabulary may be longer
    assert _backward(L, B=3, D=8, V=2**31 - 513, gw=None) == bd.FS_ERR_HIP
