"""The log-sum-exp beside a target of next to no probability (GPU): it is the other
rows', with their accuracy, however far below them the target's logit lies.

With the target's share below 2^-100 the log-sum-exp of all rows is that of the others:
off by e (a logit's error, of the rows without the far entry) and 2^-22 of values of its
size, as in test_gpu_token_logprobs.  The far logit itself, and with it the target's
log-probability, is a sum whose partial sums have the far entry's size x: each of its D
additions rounds by up to 2^-24 x, independently, which is logit_tolerance of its row
(far_error: 4 * 2^-24 sqrt(D) x; 1e-3 for x = 2^10 and D = 2048)."""
import pytest
import torch

import head_ref
import lm_head_exact_amd as fs
import test_gpu_cross_entropy as xent
import training_ref as ref
from test_gpu_token_logprobs import dev, make

pytestmark = pytest.mark.gpu

FAR = [-2.0 ** 10, -2.0 ** 20, -2.0 ** 100]


def far_error(h, W, T):
    return ref.logit_tolerance(h, W[W.shape[0] // 2:][:1], T)


@pytest.mark.parametrize("B,D,V", [(5, 1024, 700), (32, 2048, 300), (40, 128, 803), (60, 72, 803), (500, 96, 2001)])
@pytest.mark.parametrize("far", FAR)
def test_token_logprobs(B, D, V, far):
    h, W, T, ids = make(B, D, V, seed=51, ignore=0.0)
    h[:, 1], W[V // 2, 1], ids[:] = 1.0, far, V // 2
    lp, lse = (x.cpu().double() for x in fs.token_logprobs(*dev(h, W, T, ids)))
    keep = torch.arange(V) != V // 2
    e = ref.logit_tolerance(h, W[keep], T)
    want = torch.logsumexp(ref.scaled_logits(h, W[keep], T), dim=1)
    assert ((lse - want).abs() <= e + 2.0 ** -22 * (1 + want.abs())).all(), float((lse - want).abs().max())
    want_lp = ref.scaled_logits(h, W, T)[:, V // 2] - want
    # the far logit is rounded twice, its difference to the others and the result once each
    assert ((lp - want_lp).abs() <= e + far_error(h, W, T) + 2.0 ** -22 * (1 + want_lp.abs())).all()


@pytest.mark.parametrize("B,D,V", [(5, 64, 300), (90, 64, 300), (300, 72, 500), (600, 64, 500), (600, 264, 500)])
@pytest.mark.parametrize("far", FAR[:2])
@pytest.mark.parametrize("z_loss", [0.0, 1e-2])
def test_cross_entropy(B, D, V, far, z_loss):
    """Loss, statistics and gradients, whose probabilities are taken from the log-sum-exp."""
    h, W, t = xent.make(B, D, V, seed=52)
    t[t == V // 2] = 0
    t[::4] = V // 2
    h[:, 1], W[V // 2, 1] = 1.0, far
    e = ref.logit_tolerance(h, W[torch.arange(V) != V // 2], None)
    want = head_ref.cross_entropy(h, W, t, z_loss=z_loss)
    for grads in (True, False):
        stats, losses, gh, gw = xent.run(h, W, t, z_loss=z_loss, need_h=grads, need_W=grads)
        rows = t == V // 2
        err = (losses.cpu().double() - want["losses"]).abs()[rows]
        lse, nll = want["lse"].abs()[rows], want["nll"][rows]
        tol = 2 * e + far_error(h, W, None) + 2.0 ** -21 * (1 + nll) + z_loss * (2 * lse * e + 2.0 ** -21 * lse ** 2)
        assert (err <= tol).all()
        own = losses.cpu().double()[t >= 0].mean()
        assert abs(float(stats[0]) - float(own)) <= 2.0 ** -23 * float(own)
        # the other rows, the mean squared log-sum-exp and the gradients
        losses, stats = losses.clone(), stats.clone()
        losses[rows.cuda()] = want["losses"][rows].float().cuda()
        stats[:2] = want["stats"][:2].float().cuda()
        xent.check(h, W, t, (stats, losses, gh, gw), want, z_loss=z_loss, e=e)
