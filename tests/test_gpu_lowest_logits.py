"""Logits of the type's lowest value (GPU): entries masked by a finite value, as by
torch.finfo(torch.bfloat16).min in a column of W whose hidden state is 1, have
probability 0 like those of -inf, in stretches longer than any lane's or wave's share;
and a largest one has all of it.  Compared with plain fp64 without the masked rows,
within the tolerances of the operators' tests."""
import pytest
import torch

import head_ref
import lm_head_exact_amd as fs
import test_gpu_cross_entropy as xent
import training_ref as ref
from test_gpu_logprob_infinities import SHAPES
from test_gpu_token_logprobs import check_backward, check_forward, dev, make

pytestmark = pytest.mark.gpu

LOWEST = torch.finfo(torch.bfloat16).min


def without(V, rows):
    """Which rows of W stay, and their new numbers."""
    keep = torch.ones(V, dtype=torch.bool)
    keep[rows] = False
    return keep, torch.cumsum(keep, 0).to(torch.int32) - 1


@pytest.mark.parametrize("B,D,V", SHAPES)
@pytest.mark.parametrize("count", [1, 37, 160])
@pytest.mark.parametrize("value", [LOWEST, -1e38, -2.0 ** 64])
def test_token_logprobs(B, D, V, count, value):
    """(Temperatures below 1 take the scaled logits past fp32: -inf.)"""
    h, W, T, ids = make(B, D, V, seed=61)
    rows = torch.arange(V // 3, V // 3 + count)
    h[:, D // 2], W[rows, D // 2] = 1.0, value
    ids[(ids >= V // 3) & (ids < V // 3 + count)] = 0
    keep, new = without(V, rows)
    ids2 = torch.where(ids >= 0, new[ids.clamp(min=0).long()], ids)
    hd, Wd, Td, idd = dev(h, W, T, ids)
    layouts = [fs.token_logprobs(hd, Wd, Td, idd)]
    if D % 32 == 0:
        layouts.append(fs.token_logprobs(hd, fs.pack_weights(Wd), Td, idd, V=V))
    for got in layouts:
        check_forward(h, W[keep], T, ids2, 0, got)


XENT = [(5, 64, 400), (20, 64, 400), (90, 72, 700), (300, 72, 1000), (600, 64, 1000), (600, 264, 1000)]


@pytest.mark.parametrize("B,D,V", XENT)
@pytest.mark.parametrize("count", [1, 160])
@pytest.mark.parametrize("z_loss", [0.0, 1e-2])
def test_cross_entropy(B, D, V, count, z_loss):
    h, W, t = xent.make(B, D, V, seed=62)
    rows = torch.arange(V // 3, V // 3 + count)
    h[:, 1], W[rows, 1] = 1.0, LOWEST
    t[(t >= V // 3) & (t < V // 3 + count)] = 0
    keep, new = without(V, rows)
    t2 = torch.where(t >= 0, new[t.clamp(min=0).long()], t)
    want = head_ref.cross_entropy(h, W[keep], t2, z_loss=z_loss)
    stats, losses, gh, gw = xent.run(h, W, t, z_loss=z_loss)
    xent.check(h, W[keep], t2, (stats, losses, gh, gw[keep.cuda()]), want, z_loss=z_loss)
    assert (gw[rows.cuda()] == 0).all()
    alone = xent.run(h, W, t, z_loss=z_loss, need_h=False, need_W=False)
    xent.check(h, W[keep], t2, alone, want, z_loss=z_loss)


def largest(h, W, ids, column):
    """A logit of 2^127.9 in the even hidden states, of its negative in the odd ones."""
    h, W = h.clone(), W.clone()
    V = W.shape[0]
    h[:, column] = torch.tensor([1.0, -1.0])[torch.arange(h.shape[0]) % 2].to(torch.bfloat16)
    W[V // 2, column] = -LOWEST
    return h, W, torch.where(ids == V // 2, torch.zeros_like(ids), ids)


@pytest.mark.parametrize("B,D,V", [(5, 64, 400), (20, 96, 300), (60, 72, 803), (500, 96, 2001)])
def test_a_largest_logit(B, D, V):
    """It has the probability 1 where it is positive."""
    h, W, _, ids = make(B, D, V, seed=63, temp=False)
    h, W, ids = largest(h, W, ids, 1)
    lp, lse = (x.cpu().double() for x in fs.token_logprobs(*dev(h, W, None, ids)))
    even = torch.arange(B) % 2 == 0
    top = float(torch.tensor(-LOWEST).to(torch.bfloat16))
    assert (lse[even] == top).all() and (lp[even & (ids >= 0)] == -top).all()
    keep, new = without(V, [V // 2])
    ids2 = torch.where(ids >= 0, new[ids.clamp(min=0).long()], ids)
    check_forward(h[~even], W[keep], None, ids2[~even], 0, (lp[~even], lse[~even]))
    # its gradient: all of a row's from that logit
    g = torch.ones(B) / B
    got = fs.token_logprobs_backward(*dev(h, W, None, ids, lp.float(), lse.float(), g))
    want = ref.logprobs_backward(h, W, None, ids, 0, lp.float(), lse.float(), g)
    fine = ref.logit_tolerance(h, W[keep], None)
    gw = got[1].cpu().double()[V // 2]
    assert torch.isfinite(got[1]).all()
    assert ((gw - want[1][V // 2]).abs() <= (2.0 ** -7 + fine) * want[3][V // 2]).all()
    check_backward((None, got[1].cpu()[keep]), (None, want[1][keep], None, want[3][keep]), fine + 2.0 ** -19)


@pytest.mark.parametrize("B,D,V", XENT)
def test_a_largest_logit_in_the_cross_entropy(B, D, V):
    h, W, t = xent.make(B, D, V, seed=64)
    h, W, t = largest(h, W, t, 1)
    top = float(torch.tensor(-LOWEST).to(torch.bfloat16))
    even = (torch.arange(B) % 2 == 0) & (t >= 0)
    for grads in (True, False):
        _, losses, _, gw = xent.run(h, W, t, need_h=False, need_W=grads)
        assert (losses.cpu()[even].double() == top).all()
        if grads:
            n = int((t >= 0).sum())
            want = h[even].double().sum(dim=0) / n
            size = h[even].double().abs().sum(dim=0) / n
            assert torch.isfinite(gw).all()
            assert ((gw.cpu().double()[V // 2] - want).abs() <= 2.0 ** -7 * size).all()
