"""fs_cross_entropy against plain fp64 (GPU).

Tolerances.  A logit is off by at most e (training_ref.logit_tolerance).  A
row's nll moves by twice that, relative to 1 - p <= nll where the target is
likely, plus 2^-22 of values of its size for exponentials and logarithms and half
a step of the output; smoothing adds s (2 e + 2^-21 (1 + |lse| + |mean|)) and the
penalty l (2 |lse| e + 2^-21 lse^2).  Gradients: dz is rounded to bf16 (2^-8 of
|dz|, half a step), its kept exponential to fp16 (2^-11; below 2^-29 of the
largest 2^-40 of it), its exponent is off by e and by 2^-23 |lse|, sums are fp32
(a doubled e and 2^-20) and the result is rounded to bf16 (2^-8 of it)."""
import math

import pytest
import torch

import head_ref
import lm_head_exact_amd as fs
import training_ref as ref

pytestmark = pytest.mark.gpu


def make(B, D, V, seed=0, scale=1.5, ignore=0.2):
    g = torch.Generator().manual_seed(1000 * seed + B + D + V)
    h = torch.randn(B, D, generator=g).to(torch.bfloat16)
    W = (torch.randn(V, D, generator=g) * scale / math.sqrt(D)).to(torch.bfloat16)
    t = torch.randint(0, V, (B,), generator=g)
    t[0] = V - 1
    gone = torch.rand(B, generator=g) < ignore
    t = torch.where(gone, torch.tensor([-100, -1])[torch.arange(B) % 2], t)
    return h, W, t.to(torch.int32)


def check(h, W, t, got, want, smoothing=0.0, z_loss=0.0, e=None, **_):
    stats, losses, gh, gw = got
    e = ref.logit_tolerance(h, W, None) if e is None else e
    lse, nll = want["lse"].abs(), want["nll"]
    on = (t >= 0).to(nll.device)
    tol = (2 * e + 2.0 ** -22 * (1 + nll)) * torch.clamp(nll, max=1.0) + 2.0 ** -22 * nll
    if smoothing:
        tol = tol + smoothing * (2 * e + 2.0 ** -21 * (1 + 2 * lse + want["losses"].abs()))
    tol = tol + z_loss * (2 * lse * e + 2.0 ** -21 * lse ** 2) + 2.0 ** -23 * want["losses"].abs()
    fin = torch.isfinite(want["losses"])
    err = (losses.to(nll.device).double() - want["losses"]).abs()
    assert (err[fin] <= tol[fin]).all(), float((err - tol)[fin].max())
    assert torch.equal(torch.isposinf(losses.to(nll.device)), ~fin)
    assert (losses.to(nll.device)[~on] == 0).all()
    if fin.all():
        n = max(int(on.sum()), 1)
        tol3 = [float(tol[on].sum()) / n * (1 if stats_mean(want, n) else n),
                float((tol[on]).sum()) / n if not (smoothing or z_loss) else 2 * e + 2.0 ** -20 * (1 + float(nll[on].max() if on.any() else 0)),
                float((2 * lse * (e + 2.0 ** -22 * (1 + lse)) + 2.0 ** -22 * lse ** 2)[on].sum()) / n]
        for i in range(3):
            w = float(want["stats"][i])
            if math.isinf(w):   # (the mean of lse - z_y of a target of probability 0)
                assert float(stats[i]) == w
                continue
            assert abs(float(stats[i]) - w) <= tol3[i] + 2.0 ** -23 * abs(w), (i, float(stats[i]), w)
    top = float(lse[on].max()) if on.any() else 0.0
    for x, w, bound in ((gh, want["grad_h"], want["bound_h"]), (gw, want["grad_W"], want["bound_W"])):
        if x is None:
            continue
        b = bound * (2.0 ** -8 + 2.0 ** -11 + 2 * (e + 2.0 ** -23 * top) + 2.0 ** -20)
        b = b + 2.0 ** -8 * w.abs() + 2.0 ** -40 * float(bound.max()) * 8
        err = (x.to(w.device).double() - w).abs()
        assert (err <= b).all(), float((err / b.clamp(min=1e-300)).max())


def stats_mean(want, n):
    return abs(float(want["stats"][0]) * n - float(want["losses"].sum())) <= 1e-9 * (1 + abs(float(want["losses"].sum())))


def run(h, W, t, **kw):
    args = {("label_smoothing" if k == "smoothing" else k): v for k, v in kw.items()}
    return fs.cross_entropy(h.cuda(), W.cuda(), t.cuda(), **args)


def case(h, W, t, **kw):
    args = {("label_smoothing" if k == "smoothing" else k): v for k, v in kw.items()}
    got = run(h, W, t, **kw)
    check(h, W, t, got, head_ref.cross_entropy(h, W, t, **args), **kw)
    return got


SHAPES = [(1, 8, 1), (1, 8, 17), (2, 40, 33), (5, 4096, 301), (16, 256, 1000), (17, 520, 515),
          (33, 64, 255), (64, 72, 257), (65, 128, 256), (128, 200, 511), (129, 320, 513),
          (257, 136, 1025), (300, 1096, 700)]
# one shape per tile of the logits: 256 x 64, 256 x 128, 256 x 256, 128 x 128, 64 x 64, 64 x 128
TILES = [(200, 64, 16032), (500, 72, 16001), (1000, 64, 16030), (3833, 96, 2161), (513, 136, 2001),
         (200, 32, 7000)]
# and those of more than 512 rows again with rows long enough for the exponentials to be kept
TILES += [(1000, 264, 16030), (3833, 320, 2161), (513, 328, 2001)]


@pytest.mark.parametrize("B,D,V", SHAPES)
@pytest.mark.parametrize("smoothing,z_loss,reduction", [(0.0, 0.0, "mean"), (0.1, 1e-3, "sum")])
def test_loss_and_gradients(B, D, V, smoothing, z_loss, reduction):
    case(*make(B, D, V), smoothing=smoothing, z_loss=z_loss, reduction=reduction)


@pytest.mark.parametrize("B,D,V", TILES)
@pytest.mark.parametrize("smoothing,z_loss", [(0.0, 1e-2), (0.2, 0.0)])
def test_every_tile(B, D, V, smoothing, z_loss):
    h, W, t = make(B, D, V, seed=1)
    got = case(h, W, t, smoothing=smoothing, z_loss=z_loss)
    # the loss alone: the same kernels without what they keep
    alone = run(h, W, t, smoothing=smoothing, z_loss=z_loss, need_h=False, need_W=False)
    assert alone[2] is None and alone[3] is None
    assert torch.allclose(alone[1], got[1], rtol=2.0 ** -20, atol=2.0 ** -20)


# few tiles of dW and many rows: the rows in 4, 6 and 16 parts
@pytest.mark.parametrize("B,D,V", [(1100, 136, 900), (3000, 1000, 777), (4100, 64, 300)])
@pytest.mark.parametrize("ignore", [0.0, 0.9, 1.0])
def test_rows_in_parts(B, D, V, ignore):
    h, W, t = make(B, D, V, seed=21, ignore=ignore)
    t[::3] = torch.where(t[::3] >= 0, torch.full_like(t[::3], V - 1), t[::3])   # one target many times
    got = case(h, W, t, smoothing=0.1, z_loss=1e-3)
    again = run(h, W, t, smoothing=0.1, z_loss=1e-3)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    alone = run(h, W, t, smoothing=0.1, z_loss=1e-3, need_h=False)
    assert torch.equal(alone[3], got[3])


@pytest.mark.parametrize("smoothing", [0.0, 0.1])
def test_vocabulary_in_several_slices(smoothing):
    """More vocabulary rows than a slice holds; the last one is short."""
    h, W, t = make(70, 16, 2 ** 18 + 777, seed=2)
    t[:6] = torch.tensor([0, 131071, 131072, 131327, 2 ** 18, 2 ** 18 + 776], dtype=torch.int32)
    case(h, W, t, smoothing=smoothing, z_loss=1e-3)


@pytest.mark.parametrize("smoothing", [0.0, 0.1])
def test_logits_made_twice(smoothing):
    """A batch whose exponentials are not kept: slices of dz from the row's terms.
    (The reference in fp64 on the GPU, in parts of the rows.)"""
    B, D, V = 16500, 8, 2 ** 17 + 300
    assert 2 * 16640 * (2 ** 17 + 512) > 4 << 30
    h, W, t = (x.cuda() for x in make(B, D, V, seed=3, ignore=0.5))
    kw = dict(label_smoothing=smoothing, z_loss=1e-3, reduction="sum", grad_scale=0.25)
    got = fs.cross_entropy(h, W, t, **kw)
    parts = [head_ref.cross_entropy(h[r:r + 1100], W, t[r:r + 1100], **kw) for r in range(0, B, 1100)]
    want = {k: torch.cat([p[k] for p in parts]) for k in ("losses", "lse", "nll", "grad_h", "bound_h")}
    for k in ("grad_W", "bound_W"):
        want[k] = sum(p[k] for p in parts)
    n = [int((t[r:r + 1100] >= 0).sum()) for r in range(0, B, 1100)]
    want["stats"] = torch.tensor([sum(float(p["stats"][0]) for p in parts)] +
                                 [sum(float(p["stats"][i]) * k for p, k in zip(parts, n)) / sum(n)
                                  for i in (1, 2)], dtype=torch.float64)
    e = max(ref.logit_tolerance(h[r:r + 1000], W, None) for r in range(0, 4000, 1000)) * 1.5
    check(h, W, t, got, want, smoothing=smoothing, z_loss=1e-3, e=e)


@pytest.mark.parametrize("B", [255, 256, 257, 1023, 1024, 1025, 2047, 2048])
def test_row_counts_where_kernels_change(B):
    """Places in one launch or three, and the merge of the pairs; equal targets and
    targets at the ends of the vocabulary's tiles of 256 rows."""
    h, W, t = make(B, 72, 600, seed=18, ignore=0.3)
    t[5:B:7] = torch.tensor([0, 255, 256, 511, 512, 599, -100, 17], dtype=torch.int32).repeat(B)[:len(t[5:B:7])]
    case(h, W, t, z_loss=1e-3)
    hd, Wd, td = h.cuda(), W.cuda(), t.cuda()
    _, _, gh, gw = fs.cross_entropy(hd, Wd, td, reduction="sum")
    lp, lse = fs.token_logprobs(hd, Wd, None, td)
    for need_h, need_W in ((True, True), (False, True)):
        bh, bw = fs.token_logprobs_backward(hd, Wd, None, td, lp, lse, -torch.ones_like(lp), 0, need_h, need_W)
        assert (gw.double() - bw.double()).norm() <= 2.0 ** -7 * bw.double().norm()
        assert bh is None or (gh.double() - bh.double()).norm() <= 2.0 ** -7 * bh.double().norm()


def test_nothing_carries_a_graph():
    h, W, t = (x.cuda() for x in make(8, 64, 100, seed=19))
    h.requires_grad_(True)
    assert not any(x.requires_grad for x in fs.cross_entropy(h, W, t))
    fs.cross_entropy(h, W, t)
    gh = fs.cross_entropy(h, W, t)[2]
    h.backward(gh)
    assert torch.equal(h.grad, gh)


@pytest.mark.parametrize("need_h,need_W", [(True, False), (False, True)])
def test_one_gradient(need_h, need_W):
    h, W, t = make(150, 96, 800, seed=4)
    both = run(h, W, t, smoothing=0.1)
    one = run(h, W, t, smoothing=0.1, need_h=need_h, need_W=need_W)
    assert (one[2] is None) == (not need_h) and (one[3] is None) == (not need_W)
    assert torch.equal(one[0], both[0]) and torch.equal(one[1], both[1])
    assert torch.equal(one[2] if need_h else one[3], both[2] if need_h else both[3])


@pytest.mark.parametrize("B", [1, 40, 300])
def test_rows_without_a_target(B):
    """None at all: zeros.  Some: their hidden states may be NaN."""
    h, W, t = make(B, 64, 700, seed=5, ignore=0.0)
    none = torch.full_like(t, -100)
    stats, losses, gh, gw = run(torch.full_like(h, math.nan), W, none, smoothing=0.1, z_loss=1e-3)
    assert (stats == 0).all() and (losses == 0).all() and (gh == 0).all() and (gw == 0).all()
    if B > 1:
        t[1::2] = -1
        h[1::2] = math.nan
        hz = torch.where((t >= 0)[:, None], h, torch.zeros_like(h))
        got = run(h, W, t)
        check(hz, W, t, got, head_ref.cross_entropy(hz, W, t))
        assert (got[2][1::2] == 0).all()


def test_no_rows():
    _, W, _ = make(4, 64, 300, seed=6)
    h, t = torch.empty(0, 64, dtype=torch.bfloat16), torch.empty(0, dtype=torch.int32)
    stats, losses, gh, gw = run(h, W, t)
    assert (stats == 0).all() and losses.shape == (0,) and gh.shape == (0, 64) and (gw == 0).all()
    assert (run(h, W, t, need_h=False, need_W=False)[0] == 0).all()


def test_targets_past_the_vocabulary():
    h, W, t = make(30, 64, 300, seed=7, ignore=0.2)
    t[5], t[9] = 300, 2 ** 31 - 1
    got = case(h, W, t, z_loss=1e-3)
    assert torch.isposinf(got[1][5]) and torch.isposinf(got[1][9]) and torch.isposinf(got[0][0])
    assert torch.isfinite(got[2]).all() and torch.isfinite(got[3]).all()


def test_smoothing_alone():
    """At 1 no target counts, not even one of probability 0."""
    h, W, t = make(30, 64, 300, seed=17)
    t[3], t[4] = 300, 10
    t[5] = -1
    got = case(h, W, t, smoothing=1.0, z_loss=1e-3)
    assert torch.isfinite(got[1]).all()
    got = case(h, W, torch.full_like(t, 10 ** 6), smoothing=1.0, reduction="sum")
    assert torch.isfinite(got[0][0]) and torch.isposinf(got[0][1])


def test_certain_targets_keep_their_digits():
    """Targets of probability 1 - 1e-6 and nearer to 1: loss and gradient relative to
    1 - p."""
    B, D, V = 40, 64, 500
    h, W, t = make(B, D, V, seed=8, ignore=0.0)
    w = W[t.long()].float()
    h = (w / w.norm(dim=1, keepdim=True) ** 2 * torch.linspace(18, 40, B)[:, None]).to(torch.bfloat16)
    want = head_ref.cross_entropy(h, W, t)
    assert float(want["nll"].min()) < 1e-6
    case(h, W, t)


def test_peaked_logits():
    """Logits a hundred apart: exponentials far below a tile's largest."""
    h, W, t = make(90, 64, 1200, seed=9, scale=40.0)
    case(h, W, t, smoothing=0.05, z_loss=1e-3)


@pytest.mark.parametrize("keep", [True, False])
def test_infinities_and_nan(keep):
    B, D, V = 20, 64, 400
    h, W, t = make(B, D, V, seed=10, ignore=0.0)
    t = (torch.arange(B) % 90).to(torch.int32)
    h[:, 0] = 1.0
    W[100:150, 0] = -math.inf          # logits of -inf: probability 0
    kw = dict(need_W=keep, need_h=False)
    losses = run(h, W, t, **kw)[1].cpu().double()
    rest = torch.cat([W[:100], W[150:]])
    want = head_ref.cross_entropy(h, rest, t)["losses"]
    assert (losses - want).abs().max() <= 2 * ref.logit_tolerance(h, rest, None) + 1e-5
    h[3] = math.nan                    # one row's NaN stays there
    h[4, 0] = -1.0                     # +inf among a row's logits
    losses = run(h, W, t, **kw)[1].cpu()
    bad = torch.isnan(losses)
    assert bad[3] and bad[4] and int(bad.sum()) == 2


def test_equal_calls_give_equal_bits():
    h, W, t = make(700, 128, 3000, seed=11)
    t[::3] = 5
    a = run(h, W, t, smoothing=0.1)
    for _ in range(3):
        b = run(h, W, t, smoothing=0.1)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_gradients_against_differences():
    """The loss' own differences, along random directions, against the gradients."""
    h, W, t = make(24, 64, 150, seed=12, ignore=0.0)
    kw = dict(smoothing=0.1, z_loss=1e-2, reduction="sum")
    _, _, gh, gw = run(h, W, t, **kw)
    g = torch.Generator().manual_seed(5)
    for x, grad, which in ((h, gh, 0), (W, gw, 1)):
        d = torch.randn(x.shape, generator=g)
        up, down = (x.float() + 0.02 * d).to(torch.bfloat16), (x.float() - 0.02 * d).to(torch.bfloat16)
        step = up.double() - down.double()   # what bf16 left of the direction
        lu = run(*((up, W) if which == 0 else (h, up)), t, need_h=False, need_W=False, **kw)[0][0]
        ld = run(*((down, W) if which == 0 else (h, down)), t, need_h=False, need_W=False, **kw)[0][0]
        want = float((grad.cpu().double() * step).sum())
        # bf16 gradients (2^-8, averaged over the entries) and the third differences
        assert abs(float(lu) - float(ld) - want) <= 0.01 * float((grad.cpu().double() * step).norm()) + 0.01 * abs(want)


def test_given_outputs_and_workspace():
    h, W, t = (x.cuda() for x in make(60, 64, 300, seed=13))
    want = fs.cross_entropy(h, W, t)
    n = fs.cross_entropy_workspace_bytes(60, 64, 300)
    out = (torch.full((3,), 7.0).cuda(), torch.full((60,), 7.0).cuda(), torch.full_like(h, 7.0), torch.full_like(W, 7.0))
    ws = torch.full((n,), 255, dtype=torch.uint8).cuda()
    got = fs.cross_entropy(h, W, t, out=out, workspace=ws)
    assert all(x is y for x, y in zip(got, out)) and all(torch.equal(x, y) for x, y in zip(got, want))
    alone = fs.cross_entropy_workspace_bytes(60, 64, 300, grads=False)
    assert 0 < alone < n
    with pytest.raises(fs.FlashSampleError):
        fs.cross_entropy(h, W, t, workspace=ws[:alone])
    with pytest.raises(ValueError, match="overlap"):
        fs.cross_entropy(h, W, t, out=(None, None, h, None))
    with pytest.raises(ValueError, match="overlap"):
        fs.cross_entropy(h, W, t, out=(out[1][:3], out[1], None, None))
    with pytest.raises(ValueError):
        fs.cross_entropy(h, W, t, reduction="none")
    with pytest.raises(ValueError):
        fs.cross_entropy(h, W, t[:-1])
    with pytest.raises(TypeError):
        fs.cross_entropy(h, W, t.long())
    with pytest.raises(fs.FlashSampleError):
        fs.cross_entropy(h, W, t, label_smoothing=1.5)
    with pytest.raises(fs.FlashSampleError):
        fs.cross_entropy(h, W, t, z_loss=math.nan)


def test_outputs_are_marked_as_changed():
    h, W, t = (x.cuda() for x in make(8, 64, 100, seed=14))
    gh = torch.empty_like(h)
    before = gh._version
    fs.cross_entropy(h, W, t, out=(None, None, gh, None))
    assert gh._version > before


def test_graph_replays():
    """Captured once, replayed on new inputs with eager work between."""
    h, W, t = (x.cuda() for x in make(300, 64, 1000, seed=15))
    ws = torch.empty(fs.cross_entropy_workspace_bytes(300, 64, 1000), dtype=torch.uint8, device="cuda")
    out = (torch.empty(3).cuda(), torch.empty(300).cuda(), torch.empty_like(h), torch.empty_like(W))
    kw = dict(label_smoothing=0.1, z_loss=1e-3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fs.cross_entropy(h, W, t, out=out, workspace=ws, **kw)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fs.cross_entropy(h, W, t, out=out, workspace=ws, **kw)
    for i in range(4):
        nh, nw, nt = make(300, 64, 1000, seed=20 + i, ignore=0.3 * i)
        h.copy_(nh)
        W.copy_(nw)
        t.copy_(nt)
        g.replay()
        torch.cuda.synchronize()
        want = fs.cross_entropy(h, W, t, **kw)
        assert all(torch.equal(x, y) for x, y in zip(out, want)), i


def test_two_streams_at_once():
    cases = [tuple(x.cuda() for x in make(200 + 50 * i, 64, 2000, seed=30 + i)) for i in range(2)]
    want = [fs.cross_entropy(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for s, c in zip(streams, cases):
        with torch.cuda.stream(s):
            got.append([fs.cross_entropy(*c) for _ in range(5)])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(x, y) for one in g for x, y in zip(one, w))


def test_agrees_with_the_log_probabilities():
    """The same loss through token_logprobs and its backward pass."""
    h, W, t = (x.cuda() for x in make(130, 256, 1500, seed=16))
    stats, losses, gh, gw = fs.cross_entropy(h, W, t, reduction="sum")
    lp, lse = fs.token_logprobs(h, W, None, t)
    bh, bw = fs.token_logprobs_backward(h, W, None, t, lp, lse, -torch.ones_like(lp))
    assert torch.allclose(losses, -lp, rtol=2.0 ** -20, atol=2.0 ** -22)
    for a, b in ((gh, bh), (gw, bw)):   # dz rounded apart in each, then the results
        assert (a.double() - b.double()).norm() <= 2.0 ** -7 * b.double().norm()


@pytest.mark.parametrize("B,D,V", [(1, 8, 1), (1, 8192, 40), (16, 4104, 300), (17, 1000, 2049), (32, 5120, 500),
                                   (33, 72, 700), (64, 128, 3001), (65, 64, 16), (128, 264, 5000), (129, 64, 999),
                                   (200, 136, 16032), (256, 192, 20000), (257, 64, 20000)])
@pytest.mark.parametrize("ignore", [0.0, 0.5])
def test_loss_alone(B, D, V, ignore):
    """Without gradients and smoothing few rows are scored where they lie: rows without a
    target hold NaN, a target is past the vocabulary, the workspace is just large enough."""
    h, W, t = make(B, D, V, seed=23, ignore=ignore)
    h[t < 0] = math.nan
    if ignore and B > 2:
        t[B // 2] = V
        h[B // 2] = 0.5
    hz = torch.where((t >= 0)[:, None], h, torch.zeros_like(h))
    for z_loss, reduction in ((0.0, "mean"), (1e-2, "sum")):
        kw = dict(z_loss=z_loss, reduction=reduction)
        n = fs.cross_entropy_workspace_bytes(B, D, V, False)
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        got = run(h, W, t, need_h=False, need_W=False, workspace=ws, **kw)
        check(hz, W, t, got, head_ref.cross_entropy(hz, W, t, **kw), **kw)
        again = run(h, W, t, need_h=False, need_W=False, **kw)
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    none = torch.full_like(t, -100)
    stats, losses, _, _ = run(torch.full_like(h, math.nan), W, none, need_h=False, need_W=False)
    assert (stats == 0).all() and (losses == 0).all()


@pytest.mark.parametrize("B,D,V", [(20, 512, 3000), (100, 200, 5000)])
def test_loss_alone_in_a_graph(B, D, V):
    """Replayed on new inputs, with eager work on another workspace between."""
    h, W, t = (x.cuda() for x in make(B, D, V, seed=24))
    ws = torch.empty(fs.cross_entropy_workspace_bytes(B, D, V, False), dtype=torch.uint8, device="cuda")
    out = (torch.empty(3, device="cuda"), torch.empty(B, device="cuda"), None, None)
    kw = dict(z_loss=1e-3, need_h=False, need_W=False)
    fs.cross_entropy(h, W, t, out=out, workspace=ws, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fs.cross_entropy(h, W, t, out=out, workspace=ws, **kw)
    for i in range(4):
        h2, W2, t2 = make(B, D, V, seed=25 + i, ignore=0.3 * i)
        h.copy_(h2), W.copy_(W2), t.copy_(t2)
        want = fs.cross_entropy(h, W, t, **kw)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), i
