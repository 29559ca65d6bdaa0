"""A target whose own logit is +inf has no probability (GPU): NaN, never the loss of a
perfect prediction, in the log-probabilities and in the cross entropy, whichever
kernels make them.  The batch's other rows are compared with plain fp64 within the
tolerances of their operators' tests."""
import math

import pytest
import torch

import head_ref
import lm_head_exact_amd as fs
import test_gpu_cross_entropy as xent
import training_ref as ref
from test_gpu_token_logprobs import check_forward, dev, make

pytestmark = pytest.mark.gpu


def infinite(h, W, ids, target, how):
    """Every third row has `target`, whose logit there is +inf; in the others it is -inf:
    by an infinite entry of W, or by finite ones whose sum leaves fp32."""
    h, W, ids = h.clone(), W.clone(), ids.clone()
    rows = torch.arange(h.shape[0]) % 3 == 0
    ids[rows] = target
    ids[~rows & (ids == target)] = 0
    sign = torch.where(rows, 1.0, -1.0).to(torch.bfloat16)
    if how == "entry":
        h[:, 1] = sign
        W[target, 1] = math.inf
    else:
        h[:, :4] = sign[:, None]
        W[target, :4] = 3e38
    return h, W, ids, rows


# streaming kernels, tiles of every height, row lengths that are padded
@pytest.mark.parametrize("B,D,V", [(1, 64, 40), (16, 1024, 700), (32, 2048, 300), (40, 128, 803), (60, 72, 803),
                                   (200, 64, 16032), (500, 96, 2001), (3833, 72, 2161)])
@pytest.mark.parametrize("how", ["entry", "sum"])
def test_token_logprobs(B, D, V, how):
    h, W, T, ids = make(B, D, V, seed=41)
    h, W, ids, rows = infinite(h, W, ids, V // 2, how)
    keep = torch.arange(V) != V // 2
    ids2 = torch.where(ids > V // 2, ids - 1, ids)
    some = ~rows
    hd, Wd, Td, idd = dev(h, W, T, ids)
    layouts = [fs.token_logprobs(hd, Wd, Td, idd)]
    if D % 32 == 0:
        layouts.append(fs.token_logprobs(hd, fs.pack_weights(Wd), Td, idd, V=V))
    for lp, lse in layouts:
        assert lp.cpu()[rows].isnan().all() and lse.cpu()[rows].isnan().all()
        if some.any():
            check_forward(h[some], W[keep], T[some], ids2[some], 0, (lp.cpu()[some], lse.cpu()[some]))


# the loss alone by the scoring kernels (streaming, tiles) and by its own; gradients from
# exponentials that are kept (40, 300, 600 of 264) and from logits made twice
@pytest.mark.parametrize("B,D,V,grads", [(1, 64, 40, False), (20, 512, 700, False), (100, 64, 300, False),
                                         (200, 64, 500, False), (4, 64, 300, True), (40, 64, 300, True),
                                         (300, 72, 500, True), (600, 64, 500, True), (600, 264, 500, True)])
@pytest.mark.parametrize("how", ["entry", "sum"])
def test_cross_entropy(B, D, V, grads, how):
    h, W, t = xent.make(B, D, V, seed=42, ignore=0.0)
    h, W, t, rows = infinite(h, W, t, V // 2, how)
    stats, losses, gh, gw = xent.run(h, W, t, need_h=grads, need_W=grads)
    assert losses.cpu()[rows].isnan().all() and stats.isnan().all()
    some = ~rows
    if some.any():
        keep = torch.arange(V) != V // 2
        t2 = torch.where(t > V // 2, t - 1, t)
        want = head_ref.cross_entropy(h[some], W[keep], t2[some])["losses"]
        e = ref.logit_tolerance(h[some], W[keep], None)
        tol = 2 * e + 2.0 ** -21 * (1 + want)
        assert ((losses.cpu()[some].double() - want).abs() <= tol).all()
    if grads:
        assert gh.cpu()[rows].isnan().all()


def test_weights_whose_products_leave_fp32_in_8_bits():
    """The 8-bit head's log-probabilities end in the same kernel."""
    B, D, V = 50, 128, 300
    h, W, T, ids = make(B, D, V, seed=43, temp=False, ignore=0.0)
    h, W, ids, rows = infinite(h, W, ids, V // 2, "sum")
    h[:, :4] *= 1e4
    q, s = fs.quantize_weights_fp8(W.cuda())
    for n in (B, 5):
        lp, lse = fs.token_logprobs_fp8(h[:n].cuda(), q, s, V, None, ids[:n].cuda())
        assert lp.cpu()[rows[:n]].isnan().all() and lse.cpu()[rows[:n]].isnan().all()
        assert torch.isfinite(lp.cpu()[~rows[:n]]).all()
