"""fs_policy_loss and fs_preference_loss against plain fp64 (GPU).

Tolerances.  Inputs are fp32 and exact.  A token's terms are computed in fp32
with at most 8 roundings (2^-24 each; exp adds |d| 2^-24 for its rounded
argument and one step of its own), the sums in fp64; so each entry is off by
at most (10 + |d|) 2^-24 of the sum of the absolute values of what it adds."""
import math

import pytest
import torch

import lm_head_exact_amd as fs
import training_ref as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def batch(lens, seed=0, tail=0, spread=0.3):
    g = torch.Generator().manual_seed(seed + sum(lens) + len(lens))
    cu = torch.tensor([0] + list(torch.tensor(lens, dtype=torch.long).cumsum(0)), dtype=torch.int32)
    N = int(cu[-1]) + tail
    old = -2 * torch.rand(N, generator=g) - 0.01
    lp = old + spread * torch.randn(N, generator=g)
    refp = old + 0.2 * torch.randn(N, generator=g)
    mask = torch.rand(N, generator=g) < 0.75
    return g, cu, N, lp, old, refp, mask


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


LENS = [[1], [0], [0, 0, 3], [5, 1, 0, 17, 64, 65], [4096], [300] * 14, [4097, 3], [513] * 9,
        [20000, 1, 0, 700], [70] * 130, [1000] * 40]


def check_policy(lens, seed=0, per_token=False, **kw):
    g, cu, N, lp, old, refp, mask = batch(lens, seed)
    adv = torch.randn(N if per_token else len(lens), generator=g)
    if len(adv) > 2:
        adv[1] = 0.0
    use_ref = kw.pop("use_ref", True)
    use_mask = kw.pop("use_mask", True)
    r, m = (refp if use_ref else None), (mask if use_mask else None)
    want_s, want_g = ref.policy(lp, old, adv, cu, ref=r, mask=m, per_token=per_token, **kw)
    lpd, oldd, advd, cud, rd, md = cuda(lp, old, adv, cu, r, m)
    stats, grad = fs.policy_loss(lpd, oldd, advd, cud, ref_logprob=rd, mask=md, per_token=per_token,
                                 **kw)
    stats, grad = stats.cpu().double(), grad.cpu().double()
    # |terms|: surrogate below max ratio * |A|, kl below its own value (K2, K3) or |q| (K1)
    d = float((lp - old).abs().max()) if N else 0.0
    q = float((refp - lp).abs().max()) if N else 0.0
    top = (math.exp(d) * float(adv.abs().max()) if len(adv) else 0.0) + kw.get("kl_coef", 0.0) * math.exp(q)
    tol = (10 + d + q) * U * (top + 1)
    assert ((stats - want_s).abs() <= tol * torch.tensor([2.0, 1, 1 + math.exp(q), 1])).all(), (stats, want_s)
    assert stats[3] == want_s[3].float().double()
    # each gradient: its terms times the token's weight
    n = max(1, int((mask if use_mask else torch.ones(N)).sum())) if N else 1
    w = 1.0 if kw.get("reduction") == "sequence" else 1.0 / n
    assert ((grad - want_g).abs() <= tol * w + 4 * U * want_g.abs()).all()
    return grad


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("reduction", ["token", "sequence"])
@pytest.mark.parametrize("per_token", [False, True])
def test_policy(lens, reduction, per_token):
    check_policy(lens, per_token=per_token, reduction=reduction, clip_high=0.28, kl_coef=0.1)


# more sequences than a block sums by itself, blocks and waves per sequence,
# sequences of many parts, batches around one block's
MANY = [[3] * 5000, [0, 9, 1, 0] * 1300, [700] * 600, [520] * 2100, [200000, 3], [150000, 0],
        [128] * 32, [120] * 34, [16] * 256, [9000] * 30]


@pytest.mark.parametrize("lens", MANY, ids=lambda x: f"{len(x)}x{x[0]}")
@pytest.mark.parametrize("reduction", ["token", "sequence"])
def test_policy_many(lens, reduction):
    check_policy(lens, per_token=True, reduction=reduction, clip_high=0.28, kl_coef=0.1)


@pytest.mark.parametrize("kl", ["k1", "k2", "k3"])
@pytest.mark.parametrize("dual", [0.0, 1.5])
@pytest.mark.parametrize("lens", [[40, 9], [6000, 31]])
def test_policy_kinds(kl, dual, lens):
    check_policy(lens, kl=kl, dual_clip=dual, kl_coef=0.5)


@pytest.mark.parametrize("kw", [dict(use_ref=False), dict(use_mask=False),
                                dict(use_ref=False, use_mask=False, clip_low=0.0, clip_high=0.0),
                                dict(clip_low=0.9, clip_high=10.0)])
def test_policy_optional_inputs(kw):
    check_policy([30, 0, 500, 41], **kw)


def test_policy_ratio_at_the_border():
    """log-ratios equal to log1p(clip) in fp32 lie on one side of the exact
    border; the decision is the exact one, on either side."""
    for clip in (0.2, 0.1, 0.28, 0.05):
        up, down = math.log1p(clip), math.log1p(-clip)
        near = [torch.nextafter(torch.tensor(x), torch.tensor(y)).item()
                for x in (up, down) for y in (-9.0, 9.0)] + \
               [torch.tensor(x).item() for x in (up, down)]
        lp = torch.tensor(near * 2)
        old = torch.zeros(len(lp))
        adv = torch.tensor([1.0] * len(near) + [-1.0] * len(near))
        cu = torch.tensor([0, len(lp)], dtype=torch.int32)
        want = ref.policy(lp, old, adv, cu, per_token=True, clip_low=clip, clip_high=clip)
        stats, grad = fs.policy_loss(*cuda(lp, old, adv, cu), per_token=True, clip_low=clip,
                                     clip_high=clip)
        assert torch.equal(grad.cpu() == 0, want[1] == 0), clip
        assert float(stats[3]) == want[0][3].float().item()


def test_policy_masked_tokens_may_hold_anything():
    g, cu, N, lp, old, refp, mask = batch([50, 0, 700, 3], tail=9)
    mask[50:60] = False
    mask[int(cu[3]):int(cu[4])] = False           # a sequence without any token
    adv = torch.randn(N, generator=g)
    want = ref.policy(lp, old, adv, cu, ref=refp, mask=mask, per_token=True, kl_coef=0.1,
                      reduction="sequence")
    bad = ~mask
    for x in (lp, old, refp, adv):
        x[bad] = torch.tensor([math.nan, math.inf, -math.inf, torch.finfo(torch.float32).min])[
            torch.arange(int(bad.sum())) % 4]
    grad = torch.full((N,), 123.0).cuda()
    stats, grad = fs.policy_loss(*cuda(lp, old, adv, cu), ref_logprob=refp.cuda(), mask=mask.cuda(),
                                 per_token=True, kl_coef=0.1, reduction="sequence",
                                 out=(torch.empty(4).cuda(), grad))
    end = int(cu[-1])
    assert torch.isfinite(stats).all() and (grad[end:] == 123.0).all()
    assert (grad.cpu()[:end][bad[:end]] == 0).all()
    assert torch.allclose(grad.cpu().double()[:end], want[1][:end], rtol=1e-5, atol=1e-9)


@pytest.mark.parametrize("lens", [[30, 0, 11, 8], [3000, 900, 5, 2000]])
def test_padded_batch(lens):
    """Tokens before the first and behind the last sequence: gradient 0 in a new
    tensor, left alone in a given one; their entries are not read."""
    g, cu, N, lp, old, refp, _ = batch(lens)
    front, back = 7, 300
    pad = lambda x: torch.cat([torch.full((front,), math.nan), x, torch.full((back,), math.nan)])
    adv = torch.randn(len(lens), generator=g)
    want = fs.policy_loss(*cuda(lp, old, adv, cu), ref_logprob=refp.cuda(), kl_coef=0.1)
    wantp = fs.preference_loss(*cuda(lp, cu), ref_logprob=refp.cuda())
    a = cuda(pad(lp), pad(old), adv, cu + front, pad(refp))
    stats, grad = fs.policy_loss(*a[:4], ref_logprob=a[4], kl_coef=0.1)
    _, rewards, gradp = fs.preference_loss(a[0], a[3], ref_logprob=a[4])
    assert torch.allclose(stats, want[0], rtol=1e-6) and torch.allclose(rewards, wantp[1], rtol=1e-6)
    for x, w in ((grad, want[1]), (gradp, wantp[2])):
        assert torch.allclose(x[front:front + N], w, rtol=1e-6)
        assert not x[:front].any() and not x[front + N:].any()
    # a grad of the call's own beside given statistics
    torch.full((front + N + back,), 3.0).cuda()  # (what a new tensor may find)
    grad = fs.policy_loss(*a[:4], ref_logprob=a[4], out=(torch.empty(4).cuda(), None))[1]
    assert not grad[:front].any() and not grad[front + N:].any()
    mine = torch.full((front + N + back,), 5.0).cuda()
    fs.policy_loss(*a[:4], ref_logprob=a[4], out=(torch.empty(4).cuda(), mine))
    assert (mine[:front] == 5).all() and (mine[front + N:] == 5).all()
    mine.fill_(5.0)
    fs.preference_loss(a[0], a[3], ref_logprob=a[4],
                       out=(torch.empty(3).cuda(), torch.empty(len(lens)).cuda(), mine))
    assert (mine[:front] == 5).all() and (mine[front + N:] == 5).all()


@pytest.mark.parametrize("lens", [[3, 5], [5000, 40]])
def test_nothing_counts(lens):
    g, cu, N, lp, old, refp, mask = batch(lens)
    mask[:] = False
    for red in ("token", "sequence"):
        stats, grad = fs.policy_loss(*cuda(lp, old, torch.ones(2), cu), ref_logprob=refp.cuda(),
                                     mask=mask.cuda(), kl_coef=1.0, reduction=red)
        assert not stats.any() and not grad.any()
    stats, rewards, grad = fs.preference_loss(*cuda(lp, cu), mask=mask.cuda())
    assert not stats.any() and not grad.any() and not rewards.any()


def test_no_sequences():
    cu, e = torch.zeros(1, dtype=torch.int32).cuda(), torch.empty(0).cuda()
    stats, grad = fs.policy_loss(e, e, e, cu)
    assert not stats.any() and grad.shape == (0,)
    stats, rewards, grad = fs.preference_loss(e, cu)
    assert not stats.any() and rewards.shape == (0,)
    x = torch.ones(9000).cuda()
    stats, grad = fs.policy_loss(x, x, e, cu, out=(torch.ones(4).cuda(), x.clone()))
    assert not stats.any() and (grad == 1).all()
    assert not fs.policy_loss(x, x, e, cu)[1].any()


PREFS = [[1, 1], [4, 0, 3, 7], [64, 65, 130, 1], [300] * 12, [2100, 2000], [513] * 8, [9000, 3],
         [40] * 200]


@pytest.mark.parametrize("lens", PREFS)
@pytest.mark.parametrize("kind,kw", [("sigmoid", {}), ("sigmoid", dict(label_smoothing=0.1, margin=0.5)),
                                     ("hinge", dict(margin=0.2)), ("ipo", {})])
@pytest.mark.parametrize("normalise", [False, True])
def test_preference(lens, kind, kw, normalise):
    g, cu, N, lp, old, refp, mask = batch(lens, seed=7)
    beta = 2.0 if normalise else 0.1
    kw = dict(kw, kind=kind, beta=beta, length_normalised=normalise)
    want = ref.preference(lp, cu, ref=refp, mask=mask, **kw)
    lpd, cud, rd, md = cuda(lp, cu, refp, mask)
    stats, rewards, grad = fs.preference_loss(lpd, cud, ref_logprob=rd, mask=md, **kw)
    # everything between the inputs and the outputs is fp64; each output is
    # rounded once (an fp64 sum of n terms in another order: n 2^-53 relative)
    for x, w in zip((stats, rewards, grad), want):
        err = (x.cpu().double() - w).abs()
        assert (err <= 2 * U * w.abs() + 1e-10).all(), (kind, err.max())


@pytest.mark.parametrize("lens", MANY, ids=lambda x: f"{len(x)}x{x[0]}")
@pytest.mark.parametrize("normalise", [False, True])
def test_preference_many(lens, normalise):
    test_preference(lens, "sigmoid", {}, normalise)


def test_preference_without_reference_or_mask():
    g, cu, N, lp, old, refp, mask = batch([30, 11, 25, 60])
    want = ref.preference(lp, cu, kind="sigmoid", beta=0.5, margin=0.3, length_normalised=True)
    got = fs.preference_loss(*cuda(lp, cu), beta=0.5, margin=0.3, length_normalised=True)
    for x, w in zip(got, want):
        assert ((x.cpu().double() - w).abs() <= 2 * U * w.abs() + 1e-10).all()


def test_preference_extreme_margins():
    """Log-sigmoids of +-1000 neither overflow nor lose the loss."""
    cu = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32)
    lp = torch.tensor([0.0, -1000.0, -1000.0, 0.0])
    want = ref.preference(lp, cu, beta=1.0, label_smoothing=0.1)
    got = fs.preference_loss(*cuda(lp, cu), beta=1.0, label_smoothing=0.1)
    for x, w in zip(got, want):
        assert ((x.cpu().double() - w).abs() <= 2 * U * w.abs() + 1e-10).all()


def test_gradient_scale():
    g, cu, N, lp, old, refp, mask = batch([30, 40])
    adv = torch.randn(2, generator=g)
    a = fs.policy_loss(*cuda(lp, old, adv, cu))
    b = fs.policy_loss(*cuda(lp, old, adv, cu), grad_scale=4.0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1] * 4, b[1])
    a = fs.preference_loss(*cuda(lp, cu))
    b = fs.preference_loss(*cuda(lp, cu), grad_scale=0.5)
    assert torch.equal(a[0], b[0]) and torch.equal(a[2] * 0.5, b[2])


def test_offsets_out_of_range_are_clamped():
    """Wrong offsets never reach outside the arrays (the sums are then of the
    clamped sequences)."""
    g, cu, N, lp, old, refp, mask = batch([30, 40])
    bad = torch.tensor([-5, 30, 2**31 - 1], dtype=torch.int32)
    a = fs.policy_loss(*cuda(lp, old, torch.ones(2), cu))
    b = fs.policy_loss(*cuda(lp, old, torch.ones(2), bad))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    back = torch.tensor([0, 50, 10], dtype=torch.int32)
    fs.policy_loss(*cuda(lp, old, torch.ones(2), back))
    torch.cuda.synchronize()


@pytest.mark.parametrize("lens", [[40, 9, 0, 70], [3000, 4000, 12, 500]])
def test_captured_graph(lens):
    g, cu, N, lp, old, refp, mask = batch(lens)
    lpd, oldd, cud, rd, md = cuda(lp, old, cu, refp, mask)
    adv = torch.randn(len(lens), generator=g).cuda()
    out = (torch.empty(4).cuda(), torch.empty(N).cuda())
    outp = (torch.empty(3).cuda(), torch.empty(len(lens)).cuda(), torch.empty(N).cuda())
    n = fs.loss_workspace_bytes(len(lens), N)
    ws, wp = torch.empty(n, dtype=torch.uint8).cuda(), torch.empty(n, dtype=torch.uint8).cuda()

    def step():
        fs.policy_loss(lpd, oldd, adv, cud, ref_logprob=rd, mask=md, kl_coef=0.1, out=out, workspace=ws)
        fs.preference_loss(lpd, cud, ref_logprob=rd, mask=md, out=outp, workspace=wp)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        lpd.copy_(old + 0.1 * (i + 1) * torch.randn(N, generator=g))
        md.copy_(torch.rand(N, generator=g) < 0.2 * (i + 1))
        ws.fill_(255)
        wp.fill_(17)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (*out, *outp)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (*out, *outp)))


def test_refusals():
    g, cu, N, lp, old, refp, mask = batch([30, 40])
    lp, old, cu, mask = cuda(lp, old, cu, mask)
    adv = torch.ones(2).cuda()
    for bad in (dict(kl="k4"), dict(reduction="sum"), dict(mask=mask[:5]), dict(ref_logprob=old[:5])):
        with pytest.raises(ValueError):
            fs.policy_loss(lp, old, adv, cu, **bad)
    with pytest.raises(ValueError):
        fs.policy_loss(lp, old, adv, cu, per_token=True)
    with pytest.raises(TypeError):
        fs.policy_loss(lp, old, adv, cu.long())
    with pytest.raises(fs.FlashSampleError):
        fs.policy_loss(lp, old, adv, cu, clip_low=1.5)
    with pytest.raises(ValueError):
        fs.policy_loss(lp, old, adv, cu, out=(None, lp))        # in place
    both = torch.zeros(N + 2).cuda()
    with pytest.raises(ValueError):
        fs.policy_loss(lp, old, adv, cu, out=(both[N - 2:], both[:N]))
    with pytest.raises(ValueError):
        fs.preference_loss(lp, cu, old, out=(None, None, old))
    fs.policy_loss(lp, lp, adv, cu, out=(both[-1:].new_empty(4), both[:N]))   # an input twice: fine
    with pytest.raises(ValueError):
        fs.preference_loss(lp, cu[:2])
    with pytest.raises(ValueError):
        fs.preference_loss(lp, cu, kind="logistic")
    with pytest.raises(fs.FlashSampleError):
        fs.preference_loss(lp, cu, beta=-1.0)
