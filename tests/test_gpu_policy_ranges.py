"""fs_policy_loss where its terms leave their usual range, against plain fp64
(GPU)."""
import math

import pytest
import torch

import lm_head_exact_amd as fs
import training_ref as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24

# one block; blocks or waves per sequence
LENS = [[40, 9], [6000, 31], [16] * 300]


def batch(lens, seed=0):
    g = torch.Generator().manual_seed(seed + sum(lens))
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32)
    N = int(cu[-1])
    old = -2 * torch.rand(N, generator=g) - 0.01
    lp = old + 0.3 * torch.randn(N, generator=g)
    return g, cu, N, lp, old


def run(lp, old, adv, cu, refp=None, mask=None, **kw):
    d = lambda x: None if x is None else x.cuda()
    stats, grad = fs.policy_loss(d(lp), d(old), d(adv), d(cu), ref_logprob=d(refp), mask=d(mask), **kw)
    return stats.cpu().double(), grad.cpu().double()


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("kl", ["k1", "k2", "k3"])
def test_gradient_of_far_references(lens, kl):
    """q = ref - lp from -1e30 to 80 and -inf (a reference of another shard's
    token).  Per token, with A = 1: the surrogate's term is off by at most
    (6 + |d|) 2^-24 of it (three roundings, exp's own two half steps and its
    rounded argument), the KL's by its coefficient's, its product's and its own
    roundings, 6 2^-24 of it, q's rounding (2^-24 |q|) seen through its
    derivative, their sum by 2^-24; the weight adds 2 2^-24."""
    g, cu, N, lp, old = batch(lens)
    q = torch.tensor([-1e30, -1e9, -3e7, -1e5, -100.0, -20.0, -3.0, -0.6, -0.5, -0.4, -1e-3, 0.0,
                      1e-3, 0.49, 0.51, 3.0, 20.0, 80.0, -math.inf])[torch.arange(N) % 19]
    if kl == "k2":
        q = q.clamp(min=-1e15)   # (its value, q^2 / 2, stays in range)
    refp = lp + q
    adv, coef = torch.ones(len(lens)), 0.5
    _, want = ref.policy(lp, old, adv, cu, ref=refp, kl=kl, kl_coef=coef)
    stats, grad = run(lp, old, adv, cu, refp, kl=kl, kl_coef=coef)
    q64, d = refp.double() - lp.double(), (lp.double() - old.double())
    slope, moves = {"k1": (torch.ones(N), torch.zeros(N)), "k2": (q64.abs(), q64.abs()),
                    "k3": (torch.expm1(q64).abs(), q64.abs().nan_to_num(posinf=0) * q64.exp())}[kl]
    tol = U / N * (torch.exp(d) * (9 + d.abs()) + coef * (9 * slope.double() + moves))
    assert torch.isfinite(want).all()
    assert ((grad - want).abs() <= tol).all(), float(((grad - want).abs() / tol).max())
    assert stats[2] == math.inf or kl != "k3"


@pytest.mark.parametrize("lens", LENS)
def test_infinite_log_ratios_have_their_limits(lens):
    """K3 at q = +inf (the model gives the token probability 0): the value's
    limit is +inf, the gradient's -inf."""
    g, cu, N, lp, old = batch(lens)
    refp = lp.clone()
    lp[5] = -math.inf
    stats, grad = run(lp, old, torch.ones(len(lens)), cu, refp, kl="k3", kl_coef=0.1)
    assert stats[0] == math.inf and stats[2] == math.inf and grad[5] == -math.inf
    rest = torch.arange(N) != 5
    assert torch.isfinite(grad[rest]).all()


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("kl", ["k1", "k2", "k3"])
def test_a_reference_without_a_coefficient_is_only_reported(lens, kl):
    """kl_coef = 0: loss and gradient are those without a reference, bit for bit,
    whatever the term is."""
    g, cu, N, lp, old = batch(lens)
    adv = torch.randn(len(lens), generator=g)
    alone = run(lp, old, adv, cu)
    refp = lp + 0.1
    near = run(lp, old, adv, cu, refp, kl=kl)
    assert near[0][2].isfinite() and near[0][2] != 0
    refp[3], refp[7], refp[11] = 200.0, -math.inf, math.nan
    far = run(lp, old, adv, cu, refp, kl=kl)
    for stats, grad in (near, far):
        assert torch.equal(stats[[0, 1, 3]], alone[0][[0, 1, 3]]) and torch.equal(grad, alone[1])
    assert far[0][2].isnan()


@pytest.mark.parametrize("lens", LENS + [[n, 1] for n in (10, 96, 1000, 4100, 6007)])
@pytest.mark.parametrize("reduction", ["token", "sequence"])
def test_gradient_is_rounded_once(lens, reduction):
    """Ratio 1 and advantages of small whole numbers: a token's term is exact, so
    its gradient is off by its own rounding alone, 2^-24, and the 3 2^-53 of a
    weight in fp64."""
    g, cu, N, lp, _ = batch(lens)
    adv = torch.tensor([3.0, -5.0, 7.0, -11.0, 13.0])[torch.arange(len(lens)) % 5]
    _, want = ref.policy(lp, lp, adv, cu, reduction=reduction)
    _, grad = run(lp, lp, adv, cu, reduction=reduction)
    assert ((grad - want).abs() <= want.abs() * (U + 2.0 ** -50)).all()


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("reduction", ["token", "sequence"])
def test_weights_beyond_fp32_leave_masked_tokens_at_zero(lens, reduction):
    g, cu, N, lp, old = batch(lens)
    mask = torch.rand(N, generator=g) < 0.5
    adv = torch.zeros(len(lens))
    adv[0] = 1e-30
    kw = dict(reduction=reduction, clip_low=0.9, clip_high=50.0)
    for scale in (1e60, 1e300):
        _, grad = run(lp, old, adv, cu, mask=mask, grad_scale=scale, **kw)
        assert (grad[~mask] == 0).all() and (grad[lens[0]:] == 0).all()
        assert grad[:lens[0]][mask[:lens[0]]].isinf().all() == (scale == 1e300)
    # a weight that fp32 does not hold, a gradient that it does
    _, want = ref.policy(lp, old, adv, cu, mask=mask, **kw)
    _, grad = run(lp, old, adv, cu, mask=mask, grad_scale=1e40, **kw)
    d = float((lp - old).abs().max())
    assert ((grad - want * 1e40).abs() <= (8 + d) * U * (want * 1e40).abs()).all()
