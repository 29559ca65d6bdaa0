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


def head(B=70, D=192, V=500, seed=3):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(B, D, generator=g).to(torch.bfloat16).cuda()
    W = (torch.randn(V, D, generator=g) * 1.5 / math.sqrt(D)).to(torch.bfloat16).cuda()
    ids = torch.randint(0, V, (B,), generator=g).to(torch.int32)
    ids[::5] = -1
    T = (0.5 + torch.rand(B, generator=g)).cuda()
    return h, W, T, ids.cuda(), torch.randn(B, generator=g).cuda()


@pytest.mark.parametrize("need_h,need_W", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("B", [3, 70, 300])
def test_log_probabilities_carry_their_gradient(need_h, need_W, B):
    """The graph's backward pass is the explicit call's, bit for bit."""
    h, W, T, ids, w = head(B)
    lp, lse = fs.token_logprobs(h, W, T, ids)
    want = fs.token_logprobs_backward(h, W, T, ids, lp, lse, w)
    h.requires_grad_(need_h)
    W.requires_grad_(need_W)
    got = fs.token_logprobs(h, W, T, ids)
    assert torch.equal(got[0], lp) and torch.equal(got[1], lse) and got[0].requires_grad
    (got[0] * w).sum().backward()
    for x, g, need in ((h, want[0], need_h), (W, want[1], need_W)):
        assert torch.equal(x.grad, g) if need else x.grad is None
    # a gradient in the layout of a sum's: one value, expanded
    h.grad = W.grad = None
    fs.token_logprobs(h, W, T, ids)[0].sum().backward()
    want = fs.token_logprobs_backward(h.detach(), W.detach(), T, ids, lp, lse, torch.ones_like(lp))
    for x, g, need in ((h, want[0], need_h), (W, want[1], need_W)):
        assert torch.equal(x.grad, g) if need else x.grad is None


def test_gradient_reaches_the_layers_before_and_accumulates():
    h, W, T, ids, w = head()
    layer = torch.eye(h.shape[1], dtype=torch.bfloat16, device="cuda").requires_grad_(True)
    W.requires_grad_(True)
    for times in (1, 2):
        fs.token_logprobs(h @ layer, W, T, ids)[0].backward(w)
        d = h.detach()
        lp, lse = fs.token_logprobs(d, W.detach(), T, ids)
        gh, gw = fs.token_logprobs_backward(d, W.detach(), T, ids, lp, lse, w)
        assert torch.equal(layer.grad, sum([d.t() @ gh] * times))
        assert torch.equal(W.grad, sum([gw] * times))


def test_policy_update_through_the_graph():
    """Scores with a graph, the loss's gradient, logprob.backward(grad)."""
    h, W, T, ids, w = head(90)
    cu = torch.tensor([0, 40, 90], dtype=torch.int32).cuda()
    W.requires_grad_(True)
    old = fs.token_logprobs(h, W.detach(), T, ids)[0]
    assert not old.requires_grad
    lp, lse = fs.token_logprobs(h, W, T, ids)
    stats, grad = fs.policy_loss(lp, old, w[:2], cu, mask=ids >= 0)
    assert not stats.requires_grad and not grad.requires_grad
    lp.backward(grad)
    want = fs.token_logprobs_backward(h, W.detach(), T, ids, old, lse.detach(), grad, need_h=False)[1]
    assert torch.equal(W.grad, want)


def test_no_graph_where_none_is_wanted():
    h, W, T, ids, w = head()
    W.requires_grad_(True)
    with torch.no_grad():
        assert not fs.token_logprobs(h, W, T, ids)[0].requires_grad
    with torch.inference_mode():
        assert not fs.token_logprobs(h, W, T, ids)[0].requires_grad
    out = (torch.empty(70).cuda(), torch.empty(70).cuda())
    lp, _ = fs.token_logprobs(h, W, T, ids, out=out)
    assert lp is out[0] and not lp.requires_grad
    assert not fs.token_logprobs(h, W.detach(), T, ids)[0].requires_grad


def test_gradients_that_do_not_exist_are_errors():
    h, W, T, ids, w = head()
    Wp = fs.pack_weights(W)
    h.requires_grad_(True)
    lp, lse = fs.token_logprobs(h, W, T, ids)
    with pytest.raises(RuntimeError, match="log-sum-exp"):
        (lp.sum() + lse.sum()).backward()
    lp, _ = fs.token_logprobs(h, Wp, T, ids, V=500)
    with pytest.raises(RuntimeError, match="fragment-order"):
        lp.sum().backward()
    lp, _ = fs.token_logprobs(h, W, T.clone().requires_grad_(True), ids)
    with pytest.raises(RuntimeError, match="temperatures"):
        lp.sum().backward()
    assert h.grad is None
    # what the backward pass reads has changed since
    lp, _ = fs.token_logprobs(h, W, T, ids)
    fs.clip_grad_norm([W], 1e-3)
    with pytest.raises(RuntimeError, match="inplace"):
        lp.sum().backward()
    # and the checks of arguments are the same
    with pytest.raises(TypeError):
        fs.token_logprobs(h, W, T, ids.long())
    with pytest.raises(ValueError):
        fs.token_logprobs(h, W, T[:3], ids)


def test_backward_pass_on_another_stream_runs_where_its_forward_did():
    h, W, T, ids, w = head(300)
    W.requires_grad_(True)
    lp, lse = fs.token_logprobs(h, W.detach(), T, ids)
    want = fs.token_logprobs_backward(h, W.detach(), T, ids, lp, lse, w, need_h=False)[1]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        lp, _ = fs.token_logprobs(h, W, T, ids)
    torch.cuda.current_stream().wait_stream(side)
    lp.backward(w)
    torch.cuda.synchronize()
    assert torch.equal(W.grad, want)


def test_captured_scoring_of_a_parameter_and_its_refused_backward_pass():
    """Scoring with weights that require a gradient can be captured, with an eager
    graph of theirs alive; a captured backward pass is the explicit call."""
    h, W, T, ids, w = head()
    W.requires_grad_(True)
    eager, _ = fs.token_logprobs(h, W, T, ids)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lp, lse = fs.token_logprobs(h, W, T, ids)
        gw = fs.token_logprobs_backward(h, W.detach(), T, ids, lp.detach(), lse.detach(), w,
                                        need_h=False)[1]
        del lp, lse
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lp, lse = fs.token_logprobs(h, W, T, ids)
        with pytest.raises(RuntimeError, match="captured"):
            lp.backward(w)
        gw = fs.token_logprobs_backward(h, W.detach(), T, ids, lp.detach(), lse.detach(), w,
                                        need_h=False)[1]
    for i in range(3):
        w.mul_(-0.5)
        h.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        a, b = fs.token_logprobs(h, W.detach(), T, ids)
        c = fs.token_logprobs_backward(h, W.detach(), T, ids, a, b, w, need_h=False)[1]
        torch.cuda.synchronize()
        assert torch.equal(lp.detach(), a) and torch.equal(gw, c)
    assert W.grad is None
    with pytest.raises(RuntimeError, match="inplace"):
        eager.sum().backward()      # (h has changed since)
