"""Argument checks of fs_cross_entropy (CPU only: nothing is launched, the
pointers are never touched)."""
import math
import random

import pytest

from conftest import gpu_available
from lm_head_exact_amd import binding as bd

A, WS, BIG = 0x10000, 0x20000, 1 << 60


@pytest.fixture(scope="module")
def L():
    return bd.lib()


def _xent(L, h=A, W=A, B=4, D=256, V=1000, t=A, s=0.1, z=1e-4, mean=1, scale=1.0, stats=A, losses=A,
          gh=A, gw=A, ws=WS, wsb=BIG):
    return L.fs_cross_entropy(h, W, B, D, V, t, s, z, mean, scale, stats, losses, gh, gw, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(D=12), bd.FS_ERR_INVALID_ARG), (dict(D=0), bd.FS_ERR_INVALID_ARG),
    (dict(V=0), bd.FS_ERR_INVALID_ARG), (dict(B=-1), bd.FS_ERR_INVALID_ARG),
    (dict(s=-0.1), bd.FS_ERR_INVALID_ARG), (dict(s=1.01), bd.FS_ERR_INVALID_ARG),
    (dict(s=math.nan), bd.FS_ERR_INVALID_ARG), (dict(z=-1e-9), bd.FS_ERR_INVALID_ARG),
    (dict(z=math.inf), bd.FS_ERR_INVALID_ARG), (dict(z=math.nan), bd.FS_ERR_INVALID_ARG),
    (dict(scale=math.nan), bd.FS_ERR_INVALID_ARG), (dict(scale=math.inf), bd.FS_ERR_INVALID_ARG),
    (dict(h=None), bd.FS_ERR_INVALID_ARG), (dict(W=None), bd.FS_ERR_INVALID_ARG),
    (dict(t=None), bd.FS_ERR_INVALID_ARG), (dict(stats=None), bd.FS_ERR_INVALID_ARG),
    (dict(losses=None), bd.FS_ERR_INVALID_ARG), (dict(ws=None), bd.FS_ERR_INVALID_ARG),
    (dict(h=A + 8), bd.FS_ERR_INVALID_ARG), (dict(W=A + 2), bd.FS_ERR_INVALID_ARG),
    (dict(gh=A + 8), bd.FS_ERR_INVALID_ARG), (dict(gw=A + 4), bd.FS_ERR_INVALID_ARG),
    (dict(t=A + 2), bd.FS_ERR_INVALID_ARG), (dict(stats=A + 1), bd.FS_ERR_INVALID_ARG),
    (dict(losses=A + 2), bd.FS_ERR_INVALID_ARG), (dict(ws=WS + 128), bd.FS_ERR_INVALID_ARG),
    (dict(wsb=256), bd.FS_ERR_WORKSPACE),
    (dict(B=(1 << 22) + 1), bd.FS_ERR_UNSUPPORTED), (dict(D=(1 << 20) + 8), bd.FS_ERR_UNSUPPORTED),
    (dict(V=2**31 - 512), bd.FS_ERR_UNSUPPORTED),
    (dict(B=3, D=8, V=1 << 30), bd.FS_ERR_UNSUPPORTED),
    (dict(B=0, W=None), bd.FS_ERR_INVALID_ARG),
])
def test_argument_errors(L, kw, status):
    assert _xent(L, **kw) == status
    assert b"fs_cross_entropy" in L.fs_last_error()


@pytest.mark.parametrize("B,D,V", [(1, 256, 1000), (33, 264, 1000), (4096, 4096, 128256), (0, 64, 100),
                                   (20000, 64, 128256), (100, 16, 300000)])
@pytest.mark.parametrize("grads", [0, 1])
def test_workspace_is_checked_to_the_byte(L, B, D, V, grads):
    need = L.fs_cross_entropy_workspace_bytes(B, D, V, grads)
    assert need > 0 and need % 256 == 0
    g = A if grads else None
    assert _xent(L, B=B, D=D, V=V, gh=g, gw=g, wsb=need - 1) == bd.FS_ERR_WORKSPACE


def test_workspace_sizes(L):
    f = L.fs_cross_entropy_workspace_bytes
    assert f(4, 7, 1000, 1) == 0 and f(4, 256, 0, 1) == 0 and f(-1, 256, 10, 1) == 0 and f(4, 1 << 21, 9, 1) == 0
    # exponentials are kept up to 4 GiB, then a slice of 1 GiB
    assert f(16128, 320, 128256, 1) > 2 * 16128 * 128256
    assert f(512, 64, 128256, 1) > 2 * 512 * 128256
    assert f(1 << 17, 64, 128256, 1) < 2 * (1 << 17) * 128256 // 4
    # none of it for the loss alone
    assert f(4096, 64, 128256, 0) < 2 * 4096 * 128256 // 8


def test_injected_launch_failure(L, monkeypatch):
    monkeypatch.setenv("FS_FAULT_INJECT", "launch")
    assert _xent(L) == bd.FS_ERR_HIP
    assert b"FS_FAULT_INJECT" in L.fs_last_error()
    # sizes within the stated limits are taken
    r = random.Random(4)
    sizes = [(3, 8, (1 << 30) - 256), (1 << 22, 8, 1), (1 << 22, 1 << 16, 128256), (1, 1 << 20, 1 << 29)]
    sizes += [(int(2 ** r.uniform(0, 22)), 8 * int(2 ** r.uniform(0, 17)), int(2 ** r.uniform(0, 29.999)))
              for _ in range(1000)]
    for B, D, V in sizes:
        if B * D <= 2**38:
            assert _xent(L, B=B, D=D, V=V) == bd.FS_ERR_HIP, (B, D, V)
            assert _xent(L, B=B, D=D, V=V, gh=None, gw=None) == bd.FS_ERR_HIP, (B, D, V)


@pytest.mark.skipif(gpu_available(), reason="needs a machine without a GPU")
def test_launch_without_a_device_reports_the_runtime_error(L, monkeypatch):
    monkeypatch.delenv("FS_FAULT_INJECT", raising=False)
    assert _xent(L) == bd.FS_ERR_HIP
    assert b"FS_FAULT_INJECT" not in L.fs_last_error()


def test_binding_refuses_host_tensors():
    import torch
    h, W = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(5, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bd.cross_entropy(h, W, torch.zeros(2, dtype=torch.int32))
