"""The training operators one after another, as a policy or preference update
runs them: sample from the head, score under old, reference and current
weights, loss, gradients of the head and the hidden states, clipping -- against
the same chain in fp64, and captured into one graph (GPU)."""
import math
import threading

import pytest
import torch

import lm_head_exact_amd as fs
import training_ref as ref

pytestmark = pytest.mark.gpu

D, V = 192, 700


def setup(lens, seed=0):
    g = torch.Generator().manual_seed(seed)
    N = sum(lens)
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32)
    h = torch.randn(N, D, generator=g).to(torch.bfloat16)
    W = (torch.randn(V, D, generator=g) * 1.3 / math.sqrt(D))
    new = (W + 0.02 * torch.randn(V, D, generator=g) / math.sqrt(D)).to(torch.bfloat16)
    W = W.to(torch.bfloat16)
    T = torch.full((N,), 0.8)
    prompt = torch.rand(N, generator=g) < 0.3
    return g, cu, h, W, new, T, prompt


def sample(h, W, T):
    ids, _ = fs.sample(h, W, T, 11, 3)
    old, _ = fs.token_logprobs(h, fs.pack_weights(W), T, ids, V=V)
    return ids, old


def check_grads(got, h, W, T, ids, lp, lse, glp, g_tol, scale):
    """grad_h, grad_W against the fp64 chain; g_tol: relative error of glp."""
    want = ref.logprobs_backward(h, W, T, ids, 0, lp.float(), lse.float(), glp)
    e = ref.logit_tolerance(h, W, T) + 2.0 ** -22 * float(lse.abs().max()) + g_tol
    for x, w, bound in ((got[0], want[0], want[2]), (got[1], want[1], want[3])):
        # dz rounded to bf16 (2^-8), the result rounded twice: by the product and by the clipping
        tol = scale * (bound * (2.0 ** -8 + 4 * e + 2.0 ** -18) + 2 * 2.0 ** -8 * w.abs())
        err = (x.cpu().double() - scale * w).abs()
        assert (err <= tol).all(), float((err / tol.clamp(min=1e-300)).max())


@pytest.mark.parametrize("lens", [[7, 1, 0, 30], [130, 64, 200]])
@pytest.mark.parametrize("reduction", ["token", "sequence"])
def test_policy_update(lens, reduction):
    g, cu, h, W, new, T, prompt = setup(lens)
    N, S = h.shape[0], len(lens)
    hd, Wd, nd, Td = h.cuda(), W.cuda(), new.cuda(), T.cuda()
    ids, old = sample(hd, Wd, Td)
    mask = ~prompt
    targets = torch.where(prompt.cuda(), torch.full_like(ids, -1), ids)
    adv = torch.randn(S, generator=g)
    refp = fs.token_logprobs(hd, Wd, Td, targets)[0]
    lp, lse = fs.token_logprobs(hd, nd, Td, targets)
    kw = dict(kl_coef=0.05, reduction=reduction, clip_high=0.3)
    stats, glp = fs.policy_loss(lp, old, adv.cuda(), cu.cuda(), ref_logprob=refp, mask=mask.cuda(), **kw)
    gh, gw = fs.token_logprobs_backward(hd, nd, Td, targets, lp, lse, glp)
    norm = fs.clip_grad_norm([gh, gw], 0.01)

    # the same in fp64 from the sampled tokens
    ids_c = torch.where(prompt, torch.full_like(ids.cpu(), -1), ids.cpu())
    old64, _ = ref.logprobs(h, W, T, ids.cpu(), 0)
    ref64, _ = ref.logprobs(h, W, T, ids_c, 0)
    lp64, lse64 = ref.logprobs(h, new, T, ids_c, 0)
    s64, g64 = ref.policy(lp64, old64, adv, cu, ref=ref64, mask=mask, **kw)
    e = 4 * ref.logit_tolerance(h, new, T) + 2.0 ** -20
    assert ((stats.cpu().double() - s64).abs() <= e * (1 + s64.abs()) * 4).all()
    assert ((glp.cpu().double() - g64).abs() <= 8 * e * g64.abs().max()).all()
    want = ref.logprobs_backward(h, new, T, ids_c, 0, lp64.float(), lse64.float(), g64)
    n64 = math.sqrt(float((want[0] ** 2).sum() + (want[1] ** 2).sum()))
    assert abs(float(norm) - n64) <= 2.0 ** -8 * n64 + 8 * e * n64
    check_grads((gh, gw), h, new, T, ids_c, lp64, lse64, glp.cpu(), 8 * e, min(1.0, 0.01 / (n64 + 1e-6)))


def test_preference_update():
    lens = [20, 33, 5, 41, 12, 9]
    g, cu, h, W, new, T, prompt = setup(lens, seed=3)
    hd, Wd, nd = h.cuda(), W.cuda(), new.cuda()
    ids, _ = sample(hd, Wd, T.cuda())
    targets = torch.where(prompt.cuda(), torch.full_like(ids, -1), ids)
    refp, _ = fs.token_logprobs(hd, Wd, None, targets)
    lp, lse = fs.token_logprobs(hd, nd, None, targets)
    stats, rewards, glp = fs.preference_loss(lp, cu.cuda(), ref_logprob=refp, mask=(~prompt).cuda(),
                                             beta=0.3)
    gh, gw = fs.token_logprobs_backward(hd, nd, None, targets, lp, lse, glp)
    ids_c = targets.cpu()
    ref64, _ = ref.logprobs(h, W, None, ids_c, 0)
    lp64, lse64 = ref.logprobs(h, new, None, ids_c, 0)
    s64, r64, g64 = ref.preference(lp64, cu, ref=ref64, mask=~prompt, beta=0.3)
    e = ref.logit_tolerance(h, new, None) * 2 * max(lens) + 2.0 ** -20
    assert ((stats.cpu().double() - s64).abs() <= e).all()
    assert ((rewards.cpu().double() - r64).abs() <= e).all()
    assert ((glp.cpu().double() - g64).abs() <= e * g64.abs().max()).all()
    check_grads((gh, gw), h, new, None, ids_c, lp64, lse64, glp.cpu(), e, 1.0)


def test_whole_step_in_one_graph():
    """Scoring, loss, gradients, clipping and the update of the weights as one
    captured graph, replayed with other rollouts, against the eager step."""
    lens = [60, 3, 90, 47]
    g, cu, h, W, new, T, prompt = setup(lens, seed=5)
    N = h.shape[0]
    hd, Td, cud = h.cuda(), T.cuda(), cu.cuda()
    ids = torch.randint(0, V, (N,), generator=g).to(torch.int32).cuda()
    old = -torch.rand(N, generator=g).cuda() * 4
    adv = torch.randn(len(lens), generator=g).cuda()
    mask = (~prompt).cuda()
    weights = new.cuda()
    master = weights.float()

    def step(w, m):
        lp, lse = fs.token_logprobs(hd, w, Td, ids)
        stats, glp = fs.policy_loss(lp, old, adv, cud, mask=mask)
        gh, gw = fs.token_logprobs_backward(hd, w, Td, ids, lp, lse, glp)
        norm = fs.clip_grad_norm([gh, gw], 0.05)
        m.sub_(gw, alpha=0.1)
        w.copy_(m)
        return stats, norm, gh, gw
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    w0, m0 = weights.clone(), master.clone()
    with torch.cuda.stream(side):
        step(w0, m0)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    wg, mg = weights.clone(), master.clone()
    with torch.cuda.graph(graph):
        out = step(wg, mg)
    we, me = weights.clone(), master.clone()
    wg.copy_(weights)
    mg.copy_(master)
    for i in range(4):
        ids.copy_(torch.randint(-50, V, (N,), generator=g).to(torch.int32))
        old.copy_(-torch.rand(N, generator=g) * 4)
        mask.copy_(torch.rand(N, generator=g) < 0.7)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        want = step(we, me)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        assert torch.equal(wg, we) and torch.equal(mg, me)


def test_calls_of_several_host_threads():
    """Each thread on its own stream, outputs and workspaces its own: the bits of
    a call by itself."""
    g = torch.Generator().manual_seed(21)
    B, D, V = 300, 264, 5000
    h = torch.randn(B, D, generator=g).to(torch.bfloat16).cuda()
    W = (0.1 * torch.randn(V, D, generator=g)).to(torch.bfloat16).cuda()
    ids = torch.randint(0, V, (B,), generator=g).to(torch.int32).cuda()
    cu = torch.tensor([0, 100, 300], dtype=torch.int32).cuda()
    old, adv = torch.full((B,), -9.0).cuda(), torch.tensor([1.0, -1.0]).cuda()

    def step():
        lp, lse = fs.token_logprobs(h, W, None, ids)
        stats, grad = fs.policy_loss(lp, old, adv, cu)
        gh, gw = fs.token_logprobs_backward(h, W, None, ids, lp, lse, grad)
        return lp, lse, stats, grad, gh, gw, fs.clip_grad_norm([gh, gw], 0.5)

    want = step()
    torch.cuda.synchronize()
    same = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            ok = True
            for _ in range(10):
                got = step()
                torch.cuda.current_stream().synchronize()
                ok = ok and all(torch.equal(a, b) for a, b in zip(got, want))
            torch.cuda.current_stream().synchronize()
        same.append(ok)

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert same == [True] * 3
