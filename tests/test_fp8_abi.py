"""Argument checks of the 8-bit head's entry points (CPU only: nothing is launched,
the pointers are never touched)."""
import pytest

from conftest import gpu_available
from lm_head_exact_amd import binding as bd

A, WS, BIG = 0x10000, 0x20000, 1 << 60


@pytest.fixture(scope="module")
def L():
    return bd.lib()


def _quantize(L, W=A, V=1000, D=256, packed=1, q=A, qb=BIG, scale=A):
    return L.fs_quantize_weights_fp8(W, V, D, packed, q, qb, scale, None)


def _pack(L, q=A, V=1000, D=256, out=A, ob=BIG):
    return L.fs_pack_weights_fp8(q, V, D, out, ob, None)


def _logits(L, h=A, W=A, scale=A, B=4, D=256, V=1000, f32=1, out=A, pitch=None, ws=WS, wsb=BIG, off=0):
    return L.fs_logits_fp8(h, W, scale, B, D, V, f32, out, V if pitch is None else pitch, ws, wsb, None)


def _logprobs(L, h=A, W=A, scale=A, B=4, D=256, V=1000, off=0, T=A, ids=A, lp=A, lse=A, ws=WS, wsb=BIG):
    return L.fs_token_logprobs_fp8(h, W, scale, B, D, V, off, T, ids, lp, lse, ws, wsb, None)


def _sample(L, h=A, W=A, scale=A, B=4, D=256, V=1000, off=0, T=A, ids=A, val=A, ws=WS, wsb=BIG):
    return L.fs_sample_fp8(h, W, scale, B, D, V, off, T, 1, 2, ids, val, ws, wsb, None)


PRODUCTS = {"fs_logits_fp8": _logits, "fs_token_logprobs_fp8": _logprobs, "fs_sample_fp8": _sample}


@pytest.mark.parametrize("name", PRODUCTS)
@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), bd.FS_ERR_INVALID_ARG), (dict(D=32), bd.FS_ERR_INVALID_ARG),
    (dict(D=96), bd.FS_ERR_INVALID_ARG), (dict(D=0), bd.FS_ERR_INVALID_ARG),
    (dict(V=0), bd.FS_ERR_INVALID_ARG), (dict(D=16384 + 64), bd.FS_ERR_UNSUPPORTED),
    (dict(V=2**31 - 512), bd.FS_ERR_UNSUPPORTED), (dict(B=(1 << 22) + 1), bd.FS_ERR_UNSUPPORTED),
    (dict(B=1 << 22, V=1 << 30), bd.FS_ERR_UNSUPPORTED),
    (dict(h=None), bd.FS_ERR_INVALID_ARG), (dict(W=None), bd.FS_ERR_INVALID_ARG),
    (dict(scale=None), bd.FS_ERR_INVALID_ARG), (dict(ws=None), bd.FS_ERR_INVALID_ARG),
    (dict(h=A + 8), bd.FS_ERR_INVALID_ARG), (dict(W=A + 4), bd.FS_ERR_INVALID_ARG),
    (dict(ws=WS + 64), bd.FS_ERR_INVALID_ARG), (dict(wsb=64), bd.FS_ERR_WORKSPACE),
    (dict(B=0, h=None, W=None, scale=None, ws=None), bd.FS_OK),
])
def test_argument_errors(L, name, kw, status):
    assert PRODUCTS[name](L, **kw) == status
    if status != bd.FS_OK:
        assert name.encode() in L.fs_last_error()


@pytest.mark.parametrize("call,kw", [
    (_logits, dict(out=None)), (_logits, dict(out=A + 2)), (_logits, dict(f32=0, out=A + 1)),
    (_logits, dict(pitch=999)), (_logits, dict(pitch=-1)), (_logits, dict(pitch=1 << 41)),
    (_logprobs, dict(off=-1)), (_logprobs, dict(off=2**31 - 1000)), (_logprobs, dict(ids=None)),
    (_logprobs, dict(lp=None)), (_logprobs, dict(lse=None)), (_logprobs, dict(T=A + 2)),
    (_logprobs, dict(ids=A + 1)), (_logprobs, dict(lse=A + 2)),
    (_sample, dict(off=-4)), (_sample, dict(off=2)), (_sample, dict(off=2**31 - 1000)),
    (_sample, dict(T=None)), (_sample, dict(ids=None)), (_sample, dict(val=None)),
    (_sample, dict(T=A + 1)), (_sample, dict(val=A + 2)),
    (_quantize, dict(D=250)), (_quantize, dict(D=72)), (_quantize, dict(packed=0, D=12)),
    (_quantize, dict(V=0)), (_quantize, dict(W=None)), (_quantize, dict(q=None)),
    (_quantize, dict(scale=None)), (_quantize, dict(W=A + 8)), (_quantize, dict(q=A + 8)),
    (_pack, dict(D=96)), (_pack, dict(V=0)), (_pack, dict(q=None)), (_pack, dict(out=None)),
    (_pack, dict(out=A + 4)), (_pack, dict(q=A + 8)),
])
def test_errors_of_one_call(L, call, kw):
    assert call(L, **kw) == bd.FS_ERR_INVALID_ARG
    assert len(L.fs_last_error()) > 0


def test_sizes(L):
    f = L.fs_fp8_weights_bytes
    assert f(1000, 256, 0) == 256000 and f(1000, 256, 1) == 1008 * 256 and f(16, 64, 1) == 1024
    assert f(5, 8, 0) == 40 and f(5, 8, 1) == 0 and f(0, 64, 1) == 0 and f(5, 12, 0) == 0
    assert f(5, 1 << 15, 1) == 0 and f(2**31 - 513, 64, 1) == (2**31 - 512) * 64
    assert _quantize(L, qb=1008 * 256 - 1) == bd.FS_ERR_WORKSPACE
    assert _quantize(L, packed=0, qb=255999) == bd.FS_ERR_WORKSPACE
    assert _pack(L, ob=1008 * 256 - 1) == bd.FS_ERR_WORKSPACE
    w = L.fs_fp8_workspace_bytes
    assert w(4, 96, 10) == 0 and w(-1, 64, 10) == 0 and w(4, 64, 0) == 0 and w(1, 1 << 15, 10) == 0


@pytest.mark.parametrize("B,D,V", [(1, 256, 1000), (32, 5120, 128256), (33, 320, 1000), (17, 8192, 5),
                                   (4096, 4096, 128256), (300, 16384, 777)])
def test_workspace_is_checked_to_the_byte(L, B, D, V):
    need = L.fs_fp8_workspace_bytes(B, D, V)
    assert need > 0 and need % 256 == 0
    for call in PRODUCTS.values():
        assert call(L, B=B, D=D, V=V, wsb=need - 1) == bd.FS_ERR_WORKSPACE


def test_injected_launch_failure(L, monkeypatch):
    monkeypatch.setenv("FS_FAULT_INJECT", "launch")
    for call in (_quantize, _pack, *PRODUCTS.values()):
        assert call(L) == bd.FS_ERR_HIP
        assert b"FS_FAULT_INJECT" in L.fs_last_error()
    for D in range(64, 16384 + 1, 64):   # every row length has a tile whose LDS holds its scales
        for B in (1, 20, 40, 200, 3000):
            assert _logits(L, B=B, D=D, V=128256) == bd.FS_ERR_HIP


@pytest.mark.skipif(gpu_available(), reason="needs a machine without a GPU")
@pytest.mark.parametrize("call", [_quantize, _pack, _logits, _logprobs, _sample])
def test_launch_without_a_device_reports_the_runtime_error(L, call, monkeypatch):
    monkeypatch.delenv("FS_FAULT_INJECT", raising=False)
    assert call(L) == bd.FS_ERR_HIP
    assert b"FS_FAULT_INJECT" not in L.fs_last_error()


def test_binding_refuses_host_tensors():
    import torch
    h = torch.zeros(2, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(1024, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.zeros(1, 1).to(torch.float8_e8m0fnu)
    for call in (lambda: bd.quantize_weights_fp8(h), lambda: bd.pack_weights_fp8(q.view(16, 64)),
                 lambda: bd.logits_fp8(h, q, s, 16),
                 lambda: bd.token_logprobs_fp8(h, q, s, 16, None, torch.zeros(2, dtype=torch.int32)),
                 lambda: bd.sample_fp8(h, q, s, 16, torch.ones(2), 1, 2)):
        with pytest.raises(ValueError):
            call()
