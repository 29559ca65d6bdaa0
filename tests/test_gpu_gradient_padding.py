"""Gradients of W's rows whose logits are all -inf (GPU): they have probability 0, so
the gradient of grad_W there is 0, whatever the number of rows that have a token: the
places that fill a tile's last rows have hidden states of 0, which an infinite entry
of W would turn to NaN."""
import math

import pytest
import torch

import lm_head_exact_amd as fs
import test_gpu_cross_entropy as xent
import head_ref
from test_gpu_token_logprobs import check_backward, dev, make
import training_ref as ref

pytestmark = pytest.mark.gpu

# rows that fill tiles of 16, 32 and 64 places, and that do not; D of 256 and less with more
# than 512 rows makes the logits twice, the others keep their exponentials
ROWS = [(1, 64), (15, 64), (16, 64), (17, 64), (31, 72), (32, 64), (48, 64), (63, 64), (64, 64), (65, 72), (300, 64),
        (511, 64), (528, 64), (600, 264), (640, 264), (650, 64), (1025, 72)]


@pytest.mark.parametrize("B,D", ROWS)
@pytest.mark.parametrize("ignore", [0.0, 0.3])
@pytest.mark.parametrize("smoothing", [0.0, 0.1])
def test_cross_entropy(B, D, ignore, smoothing):
    V = 900
    h, W, t = xent.make(B, D, V, seed=71, ignore=ignore)
    h[:, 2], W[100:150, 2] = 1.0, -math.inf
    t[(t >= 100) & (t < 150)] = 0
    gw = xent.run(h, W, t, need_h=False, smoothing=smoothing)[3].cpu()
    keep = torch.ones(V, dtype=torch.bool)
    keep[100:150] = False
    if smoothing:   # each loses smoothing / V of every row
        n = max(int((t >= 0).sum()), 1)
        want = -smoothing / V * h[t >= 0].double().sum(dim=0) / n
        size = smoothing / V * h[t >= 0].double().abs().sum(dim=0) / n
        assert ((gw[~keep].double() - want).abs() <= 2.0 ** -7 * size).all()
        return
    assert (gw[~keep] == 0).all()
    want = head_ref.cross_entropy(h, W[keep], torch.where(t >= 150, t - 50, t))
    e = ref.logit_tolerance(h, W[keep], None)
    tol = want["bound_W"] * (2.0 ** -8 + 2.0 ** -11 + 2 * e + 2.0 ** -19) + 2.0 ** -8 * want["grad_W"].abs()
    tol = tol + 2.0 ** -37 * float(want["bound_W"].max())
    assert ((gw[keep].double() - want["grad_W"]).abs() <= tol).all()


@pytest.mark.parametrize("B,D", ROWS)
@pytest.mark.parametrize("ignore", [0.0, 0.3])
def test_token_logprobs_backward(B, D, ignore):
    V = 900
    h, W, T, ids = make(B, D, V, seed=72, ignore=ignore)
    h[:, 2], W[100:150, 2] = 1.0, -math.inf
    ids[(ids >= 100) & (ids < 150)] = 0
    keep = torch.ones(V, dtype=torch.bool)
    keep[100:150] = False
    ids2 = torch.where(ids >= 150, ids - 50, ids)
    lp, lse = (x.float() for x in ref.logprobs(h, W[keep], T, ids2, 0))
    g = torch.randn(B, generator=torch.Generator().manual_seed(B))
    want = ref.logprobs_backward(h, W[keep], T, ids2, 0, lp, lse, g)
    _, gw = fs.token_logprobs_backward(*dev(h, W, T, ids, lp, lse, g), need_h=False)
    assert (gw.cpu()[~keep] == 0).all()
    e = ref.logit_tolerance(h, W[keep], T) + 2.0 ** -23 * float(lse.abs().max())
    check_backward((None, gw.cpu()[keep]), (None, want[1], None, want[3]), e)
