"""The policy loss's gradient per sequence, each token's within its own weight
(GPU): with the mean of sequence means a token carries 1 / (tokens of its
sequence that count x sequences that have any).

Tolerance: that of test_gpu_losses, (10 + |d| + |q|) 2^-24 of the terms'
absolute values, times the weight."""
import pytest
import torch

import lm_head_exact_amd as fs
import training_ref as ref
from test_gpu_losses import LENS, MANY, U, batch, cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", LENS + MANY, ids=lambda x: f"{len(x)}x{x[0]}")
@pytest.mark.parametrize("reduction", ["token", "sequence"])
@pytest.mark.parametrize("use_mask", [True, False])
def test_every_gradient_within_its_weight(lens, reduction, use_mask):
    g, cu, N, lp, old, refp, mask = batch(lens, seed=5)
    mask = mask if use_mask else torch.ones(N, dtype=torch.bool)
    adv = torch.randn(N, generator=g)
    kw = dict(per_token=True, reduction=reduction, clip_high=0.28, kl_coef=0.1)
    want_s, want = ref.policy(lp, old, adv, cu, ref=refp, mask=mask, **kw)
    lpd, oldd, advd, cud, rd, md = cuda(lp, old, adv, cu, refp, mask)
    stats, grad = fs.policy_loss(lpd, oldd, advd, cud, ref_logprob=rd,
                                 mask=md if use_mask else None, **kw)
    counts = torch.tensor([int(mask[a:b].sum()) for a, b in zip(cu.tolist(), cu.tolist()[1:])])
    if reduction == "token":
        w = torch.full((N,), 1.0 / max(1, int(counts.sum())), dtype=torch.float64)
    else:
        per = 1.0 / (counts.clamp(min=1).double() * max(1, int((counts > 0).sum())))
        w = per.repeat_interleave((cu[1:] - cu[:-1]).long())
    d, q = (lp - old).double(), (refp - lp).double()
    size = d.exp() * adv.double().abs() + 0.1 * (1 + q.exp())
    tol = w * (10 + d.abs() + q.abs()) * U * size
    err = (grad.cpu().double() - want).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert not grad.cpu()[~mask].any()
    # the bound is one that a gradient left out would not meet
    live = mask & (want != 0)
    assert (want.abs()[live] > tol[live]).double().mean() > 0.99 if live.any() else True
