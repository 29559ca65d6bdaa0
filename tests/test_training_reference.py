"""The fp64 references of the training operators against differences and
closed forms (CPU), so that the GPU tests rest on checked formulas."""
import math

import pytest
import torch

import training_ref as ref

F64 = torch.float64


def _batch(seed, lens):
    g = torch.Generator().manual_seed(seed)
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32)
    N = int(cu[-1])
    old = -2 * torch.rand(N, generator=g)
    return g, cu, N, old


@pytest.mark.parametrize("kl", ["k1", "k2", "k3"])
@pytest.mark.parametrize("reduction", ["token", "sequence"])
@pytest.mark.parametrize("dual", [0.0, 3.0])
def test_policy_gradient_against_differences(kl, reduction, dual):
    g, cu, N, old = _batch(3, [5, 0, 7, 1])
    lp = (old + 0.5 * torch.randn(N, generator=g)).to(F64)
    refp = old + 0.2 * torch.randn(N, generator=g)
    adv = torch.randn(4, generator=g)
    mask = torch.rand(N, generator=g) < 0.8
    kw = dict(ref=refp, mask=mask, dual_clip=dual, kl_coef=0.3, kl=kl, reduction=reduction)
    _, grad = ref.policy(lp, old, adv, cu, **kw)
    eps = 1e-6
    for t in range(N):
        e = torch.zeros(N, dtype=F64)
        e[t] = eps
        d = (ref.policy(lp + e, old, adv, cu, **kw)[0][0]
             - ref.policy(lp - e, old, adv, cu, **kw)[0][0]) / (2 * eps)
        assert abs(float(d - grad[t])) < 1e-8, t


@pytest.mark.parametrize("kind,kw", [("sigmoid", {}), ("sigmoid", dict(label_smoothing=0.2, margin=0.4)),
                                     ("hinge", dict(margin=0.3)), ("ipo", {}),
                                     ("sigmoid", dict(length_normalised=True, beta=2.0))])
def test_preference_gradient_against_differences(kind, kw):
    g, cu, N, old = _batch(4, [5, 2, 0, 7, 1, 3])
    lp = old.to(F64)
    refp = old + 0.2 * torch.randn(N, generator=g)
    kw = dict(kw, kind=kind, ref=refp, mask=torch.rand(N, generator=g) < 0.9)
    _, _, grad = ref.preference(lp, cu, **kw)
    eps = 1e-6
    for t in range(N):
        e = torch.zeros(N, dtype=F64)
        e[t] = eps
        d = (ref.preference(lp + e, cu, **kw)[0][0] - ref.preference(lp - e, cu, **kw)[0][0]) / (2 * eps)
        assert abs(float(d - grad[t])) < 1e-8, t


def test_policy_closed_forms():
    cu = torch.tensor([0, 1, 2, 3], dtype=torch.int32)
    old = torch.zeros(3)
    lp = torch.tensor([math.log(2.0), math.log(0.5), math.log(5.0)])
    adv = torch.tensor([1.0, -1.0, -1.0])
    stats, grad = ref.policy(lp, old, adv, cu, dual_clip=3.0)
    # 1.2 clipped above; 0.8 clipped below; capped at 3
    assert abs(float(stats[0]) - (-1.2 + 0.8 + 3.0) / 3) < 1e-7
    assert float(stats[3]) == 1.0 and not grad.any()


def test_preference_closed_form():
    cu = torch.tensor([0, 2, 3], dtype=torch.int32)
    stats, rewards, grad = ref.preference(torch.tensor([-1.0, -2.0, -1.0]), cu, beta=0.5)
    x = 0.5 * (-3.0 + 1.0)
    assert abs(float(stats[0]) - math.log1p(math.exp(-x))) < 1e-12
    s = 1 / (1 + math.exp(x))
    assert torch.allclose(grad, torch.tensor([-0.5 * s, -0.5 * s, 0.5 * s], dtype=F64))
    assert rewards.tolist() == [-1.5, -0.5]


def test_logprob_gradient_against_differences():
    g = torch.Generator().manual_seed(5)
    B, D, V, off = 4, 8, 13, 3
    h, W = torch.randn(B, D, generator=g, dtype=F64), torch.randn(V, D, generator=g, dtype=F64)
    T = torch.tensor([1.0, 0.5, 0.0, 2.0])
    ids = torch.tensor([off, off + 12, off + 5, -1], dtype=torch.int32)
    w = torch.randn(B, generator=g, dtype=F64)

    def f(h, W):
        return float((ref.logprobs(h, W, T, ids, off)[0] * w).sum())
    lp, lse = ref.logprobs(h, W, T, ids, off)
    gh, gw, _, _ = ref.logprobs_backward(h, W, T, ids, off, lp, lse, w)
    eps = 1e-6
    for x, gx in ((h, gh), (W, gw)):
        for i in range(x.shape[0]):
            for k in range(0, D, 3):
                e = torch.zeros_like(x)
                e[i, k] = eps
                d = (f(h + e, W) - f(h - e, W)) if x is h else (f(h, W + e) - f(h, W - e))
                assert abs(d / (2 * eps) - float(gx[i, k])) < 1e-7, (i, k)


def test_logprob_of_a_nearly_certain_token_keeps_its_accuracy():
    W = torch.tensor([[40.0], [0.0]])
    lp, lse = ref.logprobs(torch.ones(1, 1), W, None, torch.tensor([0], dtype=torch.int32), 0)
    assert abs(float(lp[0]) / -math.exp(-40.0) - 1) < 1e-12 and float(lse[0]) == 40.0


def test_clip_reference():
    norm, out = ref.clip([torch.tensor([3.0]), torch.tensor([4.0])], 1.0)
    assert norm == 5.0 and abs(float(out[1]) - 4.0 / (5.0 + 1e-6)) < 1e-12
    assert ref.clip([torch.tensor([math.inf])], 1.0)[1][0].item() == math.inf
