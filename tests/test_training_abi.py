"""Argument checks of the training operators' entry points (CPU only: nothing
is launched, the pointers are never touched)."""
import ctypes
import math

import pytest

from conftest import gpu_available
from lm_head_exact_amd import binding as bd

A = 0x10000
WS = 0x20000
BIG = 1 << 50


@pytest.fixture(scope="module")
def L():
    return bd.lib()


def _logprobs(L, fn="fs_token_logprobs", h=A, W=A, B=4, D=256, V=1000, off=0, T=A, ids=A, lp=A,
              lse=A, ws=WS, wsb=BIG):
    return getattr(L, fn)(h, W, B, D, V, off, T, ids, lp, lse, ws, wsb, None)


def _backward(L, h=A, W=A, B=4, D=256, V=1000, off=0, T=A, ids=A, lp=A, lse=A, g=A, gh=A, gw=A,
              ws=WS, wsb=BIG):
    return L.fs_token_logprobs_backward(h, W, B, D, V, off, T, ids, lp, lse, g, gh, gw, ws, wsb, None)


def _policy(L, lp=A, old=A, ref=A, adv=A, mask=A, cu=A, S=4, N=9000, per=0, lo=0.2, hi=0.2, dual=0.0,
            kc=0.1, kl=3, red=0, scale=1.0, stats=A, grad=A, ws=WS, wsb=BIG):
    return L.fs_policy_loss(lp, old, ref, adv, mask, cu, S, N, per, lo, hi, dual, kc, kl, red, scale, 0,
                            stats, grad, ws, wsb, None)


def _preference(L, lp=A, ref=A, mask=A, cu=A, P=2, N=9000, kind=0, beta=0.1, margin=0.0, eps=0.0,
                norm=0, scale=1.0, stats=A, rewards=A, grad=A, ws=WS, wsb=BIG):
    return L.fs_preference_loss(lp, ref, mask, cu, P, N, kind, beta, margin, eps, norm, scale, 1, stats,
                                rewards, grad, ws, wsb, None)


def _clip(L, grads=(A, A), out=None, numel=(100, 200), dtypes=(0, 2), n=2, max_norm=1.0, norm=A,
          ws=WS, wsb=BIG):
    g = (ctypes.c_void_p * len(grads))(*grads) if grads is not None else None
    o = (ctypes.c_void_p * len(out))(*out) if out is not None else None
    s = (ctypes.c_int64 * len(numel))(*numel) if numel is not None else None
    d = (ctypes.c_int * len(dtypes))(*dtypes) if dtypes is not None else None
    return L.fs_clip_grad_norm(g, o, s, d, n, max_norm, norm, ws, wsb, None)


@pytest.mark.parametrize("fn", ["fs_token_logprobs", "fs_token_logprobs_packed"])
@pytest.mark.parametrize("kw,status", [
    (dict(D=7), bd.FS_ERR_INVALID_ARG),
    (dict(D=0), bd.FS_ERR_INVALID_ARG),
    (dict(V=0), bd.FS_ERR_INVALID_ARG),
    (dict(B=-1), bd.FS_ERR_INVALID_ARG),
    (dict(off=-1), bd.FS_ERR_INVALID_ARG),
    (dict(off=2**31 - 1000, V=1000), bd.FS_ERR_INVALID_ARG),
    (dict(h=None), bd.FS_ERR_INVALID_ARG),
    (dict(W=None), bd.FS_ERR_INVALID_ARG),
    (dict(ids=None), bd.FS_ERR_INVALID_ARG),
    (dict(lp=None), bd.FS_ERR_INVALID_ARG),
    (dict(lse=None), bd.FS_ERR_INVALID_ARG),
    (dict(ws=None), bd.FS_ERR_INVALID_ARG),
    (dict(h=A + 8), bd.FS_ERR_INVALID_ARG),
    (dict(W=A + 2), bd.FS_ERR_INVALID_ARG),
    (dict(T=A + 2), bd.FS_ERR_INVALID_ARG),
    (dict(ids=A + 1), bd.FS_ERR_INVALID_ARG),
    (dict(ws=WS + 16), bd.FS_ERR_INVALID_ARG),
    (dict(wsb=16), bd.FS_ERR_WORKSPACE),
    (dict(B=(1 << 24) + 1), bd.FS_ERR_UNSUPPORTED),
    (dict(D=(1 << 20) + 32), bd.FS_ERR_UNSUPPORTED),
    (dict(B=1 << 24, V=2**31 - 1), bd.FS_ERR_UNSUPPORTED),
    (dict(V=2**31 - 512), bd.FS_ERR_UNSUPPORTED),
    (dict(B=0, h=None, W=None, T=None, ids=None, lp=None, lse=None, ws=None), bd.FS_OK),
])
def test_logprobs_argument_errors(L, fn, kw, status):
    assert _logprobs(L, fn, **kw) == status
    if status != bd.FS_OK:
        assert len(L.fs_last_error()) > 0


def test_logprobs_packed_needs_whole_k_steps(L):
    assert _logprobs(L, "fs_token_logprobs_packed", D=264) == bd.FS_ERR_INVALID_ARG


@pytest.mark.parametrize("B,D,V", [(1, 256, 1000), (33, 264, 1000), (4096, 4096, 128256), (17, 8192, 5)])
def test_logprobs_workspace_is_checked_to_the_byte(L, B, D, V):
    need = L.fs_token_logprobs_workspace_bytes(B, D, V)
    assert need > 0 and need % 256 == 0
    assert _logprobs(L, B=B, D=D, V=V, wsb=need - 1) == bd.FS_ERR_WORKSPACE
    back = L.fs_token_logprobs_backward_workspace_bytes(B, D, V)
    assert back > 2 * B * D
    assert _backward(L, B=B, D=D, V=V, wsb=back - 1) == bd.FS_ERR_WORKSPACE


def test_workspace_sizes_of_invalid_shapes_are_zero(L):
    for f in (L.fs_token_logprobs_workspace_bytes, L.fs_token_logprobs_backward_workspace_bytes):
        assert f(4, 7, 1000) == 0 and f(4, 256, 0) == 0 and f(-1, 256, 10) == 0 and f(4, 1 << 21, 9) == 0
    assert L.fs_loss_workspace_bytes(-1, 10) == 0 and L.fs_loss_workspace_bytes(3, -1) == 0
    s = (ctypes.c_int64 * 2)(5, -1)
    assert L.fs_clip_grad_norm_workspace_bytes(s, 2) == 0


def test_backward_workspace_stays_bounded(L):
    """dz is held for a slice of the vocabulary: 1 GiB, not B x V."""
    whole = 2 * (1 << 17) * 128256
    assert L.fs_token_logprobs_backward_workspace_bytes(1 << 17, 256, 128256) < whole // 8


@pytest.mark.parametrize("kw,status", [
    (dict(D=12), bd.FS_ERR_INVALID_ARG),
    (dict(V=0), bd.FS_ERR_INVALID_ARG),
    (dict(B=-1), bd.FS_ERR_INVALID_ARG),
    (dict(off=-1), bd.FS_ERR_INVALID_ARG),
    (dict(gh=None, gw=None), bd.FS_ERR_INVALID_ARG),
    (dict(h=None), bd.FS_ERR_INVALID_ARG),
    (dict(lp=None), bd.FS_ERR_INVALID_ARG),
    (dict(g=None), bd.FS_ERR_INVALID_ARG),
    (dict(W=A + 8), bd.FS_ERR_INVALID_ARG),
    (dict(gw=A + 8), bd.FS_ERR_INVALID_ARG),
    (dict(gh=A + 4), bd.FS_ERR_INVALID_ARG),
    (dict(lse=A + 2), bd.FS_ERR_INVALID_ARG),
    (dict(ws=WS + 8), bd.FS_ERR_INVALID_ARG),
    (dict(wsb=8), bd.FS_ERR_WORKSPACE),
    (dict(B=(1 << 22) + 1), bd.FS_ERR_UNSUPPORTED),
    (dict(D=(1 << 20) + 8), bd.FS_ERR_UNSUPPORTED),
    (dict(V=2**31 - 512), bd.FS_ERR_UNSUPPORTED),
    (dict(B=0, gw=None, h=None, W=None, ws=None), bd.FS_OK),
])
def test_backward_argument_errors(L, kw, status):
    assert _backward(L, **kw) == status
    if status != bd.FS_OK:
        assert len(L.fs_last_error()) > 0


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), bd.FS_ERR_INVALID_ARG),
    (dict(N=-1), bd.FS_ERR_INVALID_ARG),
    (dict(S=(1 << 20) + 1), bd.FS_ERR_UNSUPPORTED),
    (dict(cu=None), bd.FS_ERR_INVALID_ARG),
    (dict(cu=A + 1), bd.FS_ERR_INVALID_ARG),
    (dict(lp=None), bd.FS_ERR_INVALID_ARG),
    (dict(old=None), bd.FS_ERR_INVALID_ARG),
    (dict(adv=None), bd.FS_ERR_INVALID_ARG),
    (dict(stats=None), bd.FS_ERR_INVALID_ARG),
    (dict(grad=None), bd.FS_ERR_INVALID_ARG),
    (dict(ref=A + 2), bd.FS_ERR_INVALID_ARG),
    (dict(lo=1.0), bd.FS_ERR_INVALID_ARG),
    (dict(lo=-0.1), bd.FS_ERR_INVALID_ARG),
    (dict(lo=math.nan), bd.FS_ERR_INVALID_ARG),
    (dict(hi=-0.1), bd.FS_ERR_INVALID_ARG),
    (dict(hi=math.inf), bd.FS_ERR_INVALID_ARG),
    (dict(dual=1.0), bd.FS_ERR_INVALID_ARG),
    (dict(dual=math.nan), bd.FS_ERR_INVALID_ARG),
    (dict(kc=math.nan), bd.FS_ERR_INVALID_ARG),
    (dict(scale=math.inf), bd.FS_ERR_INVALID_ARG),
    (dict(kl=0), bd.FS_ERR_INVALID_ARG),
    (dict(red=2), bd.FS_ERR_INVALID_ARG),
    (dict(ws=None), bd.FS_ERR_INVALID_ARG),
    (dict(ws=WS + 4), bd.FS_ERR_INVALID_ARG),
    (dict(wsb=4), bd.FS_ERR_WORKSPACE),
])
def test_policy_argument_errors(L, kw, status):
    assert _policy(L, **kw) == status
    assert len(L.fs_last_error()) > 0


@pytest.mark.parametrize("kw,status", [
    (dict(P=-1), bd.FS_ERR_INVALID_ARG),
    (dict(P=1 << 24), bd.FS_ERR_UNSUPPORTED),
    (dict(N=-5), bd.FS_ERR_INVALID_ARG),
    (dict(cu=None), bd.FS_ERR_INVALID_ARG),
    (dict(lp=None), bd.FS_ERR_INVALID_ARG),
    (dict(rewards=None), bd.FS_ERR_INVALID_ARG),
    (dict(kind=3), bd.FS_ERR_INVALID_ARG),
    (dict(beta=0.0), bd.FS_ERR_INVALID_ARG),
    (dict(beta=math.inf), bd.FS_ERR_INVALID_ARG),
    (dict(beta=math.nan), bd.FS_ERR_INVALID_ARG),
    (dict(margin=math.nan), bd.FS_ERR_INVALID_ARG),
    (dict(kind=2, margin=0.1), bd.FS_ERR_INVALID_ARG),
    (dict(eps=0.6), bd.FS_ERR_INVALID_ARG),
    (dict(kind=1, eps=0.1), bd.FS_ERR_INVALID_ARG),
    (dict(grad=A + 1), bd.FS_ERR_INVALID_ARG),
    (dict(wsb=4), bd.FS_ERR_WORKSPACE),
])
def test_preference_argument_errors(L, kw, status):
    assert _preference(L, **kw) == status
    assert len(L.fs_last_error()) > 0


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), bd.FS_ERR_INVALID_ARG),
    (dict(n=65537), bd.FS_ERR_INVALID_ARG),
    (dict(grads=None), bd.FS_ERR_INVALID_ARG),
    (dict(numel=None), bd.FS_ERR_INVALID_ARG),
    (dict(numel=(100, -1)), bd.FS_ERR_INVALID_ARG),
    (dict(numel=(100, 1 << 50)), bd.FS_ERR_UNSUPPORTED),
    (dict(dtypes=(0, 3)), bd.FS_ERR_INVALID_ARG),
    (dict(grads=(A, None)), bd.FS_ERR_INVALID_ARG),
    (dict(grads=(A + 1, A)), bd.FS_ERR_INVALID_ARG),
    (dict(grads=(A, A + 2)), bd.FS_ERR_INVALID_ARG),
    (dict(out=(A, None)), bd.FS_ERR_INVALID_ARG),
    (dict(max_norm=-1.0), bd.FS_ERR_INVALID_ARG),
    (dict(max_norm=math.nan), bd.FS_ERR_INVALID_ARG),
    (dict(norm=None), bd.FS_ERR_INVALID_ARG),
    (dict(ws=WS + 4), bd.FS_ERR_INVALID_ARG),
    (dict(wsb=256), bd.FS_ERR_WORKSPACE),
])
def test_clip_argument_errors(L, kw, status):
    assert _clip(L, **kw) == status
    assert len(L.fs_last_error()) > 0


def test_small_losses_need_no_workspace(L, monkeypatch):
    monkeypatch.setenv("FS_FAULT_INJECT", "launch")
    assert L.fs_loss_workspace_bytes(4, 100) == 0 and L.fs_loss_workspace_bytes(0, 0) == 0
    assert L.fs_loss_workspace_bytes(4, 5000) > 0 and L.fs_loss_workspace_bytes(300, 300) > 0
    assert _policy(L, N=100, ws=None, wsb=0) == bd.FS_ERR_HIP        # past the checks
    assert _preference(L, N=100, ws=None, wsb=0) == bd.FS_ERR_HIP
    need = L.fs_loss_workspace_bytes(4, 9000)
    assert _policy(L, wsb=need - 1) == bd.FS_ERR_WORKSPACE
    assert _preference(L, wsb=need - 1) == bd.FS_ERR_WORKSPACE


def test_injected_launch_failure(L, monkeypatch):
    monkeypatch.setenv("FS_FAULT_INJECT", "launch")
    calls = {
        "fs_token_logprobs": lambda: _logprobs(L),
        "fs_token_logprobs_packed": lambda: _logprobs(L, "fs_token_logprobs_packed"),
        "fs_token_logprobs_backward": lambda: _backward(L),
        "fs_policy_loss": lambda: _policy(L),
        "fs_preference_loss": lambda: _preference(L),
        "fs_clip_grad_norm": lambda: _clip(L),
    }
    for name, call in calls.items():
        assert call() == bd.FS_ERR_HIP, name
        msg = L.fs_last_error()
        assert name.encode() in msg and b"FS_FAULT_INJECT" in msg, (name, msg)


@pytest.mark.skipif(gpu_available(), reason="needs a machine without a GPU")
@pytest.mark.parametrize("call", [_logprobs, _backward, _policy, _preference, _clip])
def test_launch_without_a_device_reports_the_runtime_error(L, call, monkeypatch):
    monkeypatch.delenv("FS_FAULT_INJECT", raising=False)
    assert call(L) == bd.FS_ERR_HIP
    assert len(L.fs_last_error()) > 0 and b"FS_FAULT_INJECT" not in L.fs_last_error()


def test_binding_refuses_host_tensors_and_bad_choices():
    import torch
    h, W = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(5, 8, dtype=torch.bfloat16)
    ids = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        bd.token_logprobs(h, W, None, ids)
    with pytest.raises(ValueError):
        bd.token_logprobs_backward(h, W, None, ids, *[torch.zeros(2)] * 3)
    cu = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        bd.policy_loss(torch.zeros(4), torch.zeros(4), torch.zeros(2), cu)
    with pytest.raises(ValueError):
        bd.preference_loss(torch.zeros(4), cu)
    with pytest.raises(ValueError):
        bd.clip_grad_norm([], 1.0)
    with pytest.raises(ValueError):
        bd.clip_grad_norm([torch.zeros(3)], 1.0)
    with pytest.raises(TypeError):
        bd.clip_grad_norm([torch.zeros(3, dtype=torch.int32)], 1.0)
