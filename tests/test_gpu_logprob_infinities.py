"""fs_token_logprobs where logits are infinite, against plain fp64 (GPU): a logit
of -inf has probability 0, +inf or NaN gives NaN, whichever kernel makes them
and wherever in W the infinite entry lies.

The log-sum-exps and log-probabilities are compared within the tolerances of
test_gpu_token_logprobs (a logit is off by e, the rest by 2^-22 of values of
their size)."""
import math

import pytest
import torch

import lm_head_exact_amd as fs
from test_gpu_token_logprobs import check_forward, dev, make

pytestmark = pytest.mark.gpu

# streaming kernels of one and two tiles of tokens, whole and ragged slices;
# every tile of the logits, with D a multiple of 64, of 32 and of neither
SHAPES = [(1, 1024, 700), (16, 4096, 300), (5, 1056, 300), (7, 40, 300), (32, 2048, 300), (20, 96, 300),
          (40, 128, 803), (60, 96, 803), (60, 72, 803), (200, 64, 16032), (200, 72, 16032),
          (500, 72, 16001), (500, 96, 16001), (1000, 72, 16030), (513, 136, 2001), (513, 160, 2001),
          (3833, 96, 2161), (3833, 72, 2161)]


def infinite(h, W, T, ids, off, rows, column, value):
    """W with `value` in `column` of `rows`, hidden states with +1 or -1 there: the
    rows' logits are infinite, of the sign of the product."""
    W, h = W.clone(), h.clone()
    h[:, column] = torch.tensor([1.0, -1.0])[torch.arange(h.shape[0]) % 2].to(torch.bfloat16)
    W[rows, column] = value
    return h, W


@pytest.mark.parametrize("B,D,V", SHAPES)
@pytest.mark.parametrize("where", ["first", "last"])
@pytest.mark.parametrize("count", [1, 37, 160])
def test_logits_of_minus_infinity_have_probability_zero(B, D, V, where, count):
    """Rows whose logits are -inf for the even hidden states, alone and in
    stretches longer than any lane's or wave's share; the odd ones' are +inf."""
    h, W, T, ids = make(B, D, V, seed=31)
    column = 0 if where == "first" else D - 1
    start = V // 3
    rows = torch.arange(start, start + count)
    h, W = infinite(h, W, T, ids, 0, rows, column, -math.inf)
    ids[ids >= 0] = torch.where((ids[ids >= 0] >= start) & (ids[ids >= 0] < start + count),
                                torch.zeros(1, dtype=torch.int32), ids[ids >= 0])
    even, odd = torch.arange(0, B, 2), torch.arange(1, B, 2)
    keep = torch.ones(V, dtype=torch.bool)
    keep[rows] = False
    new = torch.cumsum(keep, 0).to(torch.int32) - 1            # rows without the infinite ones
    ids2 = torch.where(ids >= 0, new[ids.clamp(min=0).long()], ids)
    Tn = None if T is None else T[even]
    layouts = [fs.token_logprobs(*dev(h, W, T, ids))]
    if D % 32 == 0:
        hd, Wd, Td, idd = dev(h, W, T, ids)
        layouts.append(fs.token_logprobs(hd, fs.pack_weights(Wd), Td, idd, V=V))
    for lp, lse in layouts:
        check_forward(h[even], W[keep], Tn, ids2[even], 0, (lp[even.cuda()], lse[even.cuda()]))
        assert lse[odd.cuda()].isnan().all()
        has = (ids[odd] >= 0).cuda()
        assert lp[odd.cuda()][has].isnan().all() and (lp[odd.cuda()][~has] == 0).all()


@pytest.mark.parametrize("B,D,V", SHAPES)
def test_target_at_minus_infinity(B, D, V):
    """Its log-probability is -inf and the log-sum-exp the others'."""
    h, W, T, ids = make(B, D, V, seed=32, ignore=0.0)
    h, W = infinite(h, W, T, ids, 0, torch.tensor([V // 2]), D // 2, -math.inf)
    h[:, D // 2] = 1.0
    ids[:] = V // 2
    keep = torch.arange(V) != V // 2
    lp, lse = fs.token_logprobs(*dev(h, W, T, ids))
    assert (lp == -math.inf).all()
    none = torch.full_like(ids, -1)
    check_forward(h, W[keep], T, none, 0, (torch.zeros(B), lse))


@pytest.mark.parametrize("B,D,V", SHAPES)
def test_every_logit_at_minus_infinity_gives_nan(B, D, V):
    h, W, T, ids = make(B, D, V, seed=33)
    h, W = infinite(h, W, T, ids, 0, torch.arange(V), 0, -math.inf)
    h[:, 0] = 1.0
    lp, lse = fs.token_logprobs(*dev(h, W, T, ids))
    assert not torch.isfinite(lse).any() and (lse < 0).logical_or(lse.isnan()).all()
    assert lp.cpu()[ids >= 0].isnan().all()


@pytest.mark.parametrize("B,D,V", [s for s in SHAPES if s[1] % 64])
def test_padding_of_rows_takes_nothing_from_infinite_entries(B, D, V):
    """Hidden states of zero where W is infinite are NaN by the product itself;
    those of +1 in the last column of an odd D see no product with padding."""
    h, W, T, ids = make(B, D, V, seed=34)
    h, W = infinite(h, W, T, ids, 0, torch.tensor([1, V - 1]), D - 1, -math.inf)
    h[:, D - 1] = 1.0
    ids[ids >= 0] = 0
    keep = torch.ones(V, dtype=torch.bool)
    keep[[1, V - 1]] = False
    check_forward(h, W[keep], T, ids, 0, fs.token_logprobs(*dev(h, W, T, ids)))
