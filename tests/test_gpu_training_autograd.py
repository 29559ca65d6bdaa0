"""The training operators among torch's autograd (GPU)."""
import math

import pytest
import torch

import lm_head_exact_amd as fs

pytestmark = pytest.mark.gpu


def saved(t):
    """A graph that has saved `t`, and the leaf behind it."""
    x = torch.ones_like(t, requires_grad=True)
    return x, (x * t).sum()


def changed(t, call):
    """Whether a graph that saved `t` before `call` refuses its backward pass."""
    x, y = saved(t)
    call()
    try:
        y.backward()
    except RuntimeError as e:
        assert "modified by an inplace operation" in str(e)
        return True
    return False


def test_tensors_that_a_call_writes_are_marked_as_changed():
    g = torch.Generator().manual_seed(1)
    a, b, c = (torch.randn(100, generator=g).cuda() for _ in range(3))
    norm = torch.zeros(1).cuda()
    assert changed(a, lambda: fs.clip_grad_norm([b, a], 0.1))
    assert changed(c, lambda: fs.clip_grad_norm([a], 0.1, out=[c]))
    assert not changed(a, lambda: fs.clip_grad_norm([a], 0.1, out=[c]))
    assert changed(norm, lambda: fs.clip_grad_norm([a], 0.1, norm=norm))
    assert not changed(a, lambda: fs.clip_grad_norm([a], math.inf))       # the norm alone

    B, D, V = 5, 64, 200
    h, W = (torch.randn(n, D, generator=g).to(torch.bfloat16).cuda() for n in (B, V))
    ids = torch.arange(B, dtype=torch.int32).cuda()
    lp, lse = torch.empty(B).cuda(), torch.empty(B).cuda()
    one = torch.ones(B).cuda()
    for t in (lp, lse):
        assert changed(t, lambda: fs.token_logprobs(h, W, None, ids, out=(lp, lse)))
    assert not changed(h, lambda: fs.token_logprobs(h, W, None, ids, out=(lp, lse)))
    gh, gw = torch.empty_like(h), torch.empty_like(W)
    for t in (gh, gw):
        assert changed(t, lambda: fs.token_logprobs_backward(h, W, None, ids, lp, lse, one, out=(gh, gw)))
    cu = torch.tensor([0, 2, 5], dtype=torch.int32).cuda()
    stats, grad, rewards = torch.empty(4).cuda(), torch.empty(B).cuda(), torch.empty(2).cuda()
    for t in (stats, grad):
        assert changed(t, lambda: fs.policy_loss(lp, one, one[:2], cu, out=(stats, grad)))
    out = (stats[:3], rewards, grad)
    for t in out:
        assert changed(t, lambda: fs.preference_loss(lp, cu, out=out))


def test_tensors_without_a_version_can_be_clipped():
    with torch.inference_mode():
        a = torch.ones(100).cuda()
        norm = fs.clip_grad_norm([a], 1.0)
        assert float(norm) == 10.0 and abs(float(a[0]) - 0.1) < 1e-6
        fs.clip_grad_norm([a], 0.5, out=[torch.empty_like(a)], norm=norm)
