"""fs_token_logprobs and its backward pass against plain fp64 (GPU).

Tolerances.  A scaled logit is off by at most e_t (training_ref.logit_tolerance).
The log-sum-exp and the log-probability move by at most that (twice for their
difference), plus the roundings of exponentials and logarithms: 2^-22 of a
value of their size plus 2^-22 for the sum's relative error.  Gradients: dz is
rounded to bf16 (2^-8 of each |dz|, half a step), its exponential is off by
e_t relative, sums are fp32 (covered by a doubled e_t) and the result is rounded
to bf16 (2^-8 of it)."""
import math

import pytest
import torch

import lm_head_exact_amd as fs
import training_ref as ref

pytestmark = pytest.mark.gpu


def make(B, D, V, off=0, seed=0, temp=True, scale=1.5, ignore=0.2):
    g = torch.Generator().manual_seed(1000 * seed + B + D + V)
    h = torch.randn(B, D, generator=g).to(torch.bfloat16)
    W = (torch.randn(V, D, generator=g) * scale / math.sqrt(D)).to(torch.bfloat16)
    T = None
    if temp:
        T = 0.4 + torch.rand(B, generator=g)
        T[3::5] = torch.tensor([0.0, -1.0, math.nan, 0.0])[torch.arange(len(T[3::5])) % 4]
    ids = torch.randint(0, V, (B,), generator=g) + off
    if off:
        ids[1::4] = torch.randint(0, off, (len(ids[1::4]),), generator=g)   # another shard's, below
        ids[2::7] = off + V + 5                                              # and above
    ids[0] = off + V - 1
    ids = torch.where(torch.rand(B, generator=g) < ignore, torch.full_like(ids, -100), ids)
    return h, W, T, ids.to(torch.int32)


def dev(*ts):
    return [None if t is None else t.cuda() for t in ts]


def check_forward(h, W, T, ids, off, got):
    lp, lse = (x.cpu().double() for x in got)
    want_lp, want_lse = ref.logprobs(h, W, T, ids, off)
    e = ref.logit_tolerance(h, W, T)
    tol = e + 2.0 ** -22 * (1 + want_lse.abs())
    assert ((lse - want_lse).abs() <= tol).all(), float((lse - want_lse).abs().max())
    fin = torch.isfinite(want_lp)
    assert torch.equal(torch.isinf(lp) & (lp < 0), ~fin)
    tol = (2 * e + 2.0 ** -22 * (1 + want_lp.abs())) * torch.clamp(want_lp.abs(), max=1.0)
    # d log p = (1 - p) d(x): relative to 1 - p <= |log p|; and half a step of the output
    tol = tol + 2.0 ** -23 * want_lp.abs()
    assert ((lp - want_lp).abs()[fin] <= tol[fin]).all(), float(((lp - want_lp).abs() - tol)[fin].max())
    assert (lp[ids < 0] == 0).all()


def backward_case(h, W, T, ids, off, seed=1, **kw):
    g = torch.Generator().manual_seed(seed)
    grad = torch.randn(h.shape[0], generator=g) / h.shape[0]
    lp, lse = ref.logprobs(h, W, T, ids, off)
    lp, lse = lp.float(), lse.float()
    want = ref.logprobs_backward(h, W, T, ids, off, lp, lse, grad)
    hd, Wd, Td, idd, lpd, lsed, gd = dev(h, W, T, ids, lp, lse, grad)
    got = fs.token_logprobs_backward(hd, Wd, Td, idd, lpd, lsed, gd, vocab_offset=off, **kw)
    return got, want, ref.logit_tolerance(h, W, T) + 2.0 ** -23 * float(lse.abs().max())


def check_backward(got, want, e):
    for x, w, bound in ((got[0], want[0], want[2]), (got[1], want[1], want[3])):
        if x is None:
            continue
        tol = bound * (2.0 ** -8 + 2 * e + 2.0 ** -20) + 2.0 ** -8 * w.abs()
        err = (x.cpu().double() - w).abs()
        assert (err <= tol).all(), float((err / tol.clamp(min=1e-300)).max())


SHAPES = [
    # streaming kernels: one and two tiles of 16 tokens, every slice length, D not a multiple of 32
    (1, 8, 1), (1, 8, 17), (2, 40, 33), (16, 256, 1000), (15, 1032, 131), (16, 2056, 95),
    (5, 4096, 301), (3, 5120, 129), (2, 6152, 65), (4, 8192, 77), (17, 512, 515), (32, 1536, 130),
    (31, 4096, 99),
    # tiles of 64, 128 and 256 tokens; ragged in every direction
    (33, 64, 255), (64, 72, 257), (65, 128, 256), (128, 200, 511), (129, 320, 513), (257, 136, 1025),
    (300, 1096, 700), (513, 64, 2000), (33, 4104, 40), (20, 8192, 50),
]


@pytest.mark.parametrize("B,D,V", SHAPES)
@pytest.mark.parametrize("off", [0, 1001])
def test_forward(B, D, V, off):
    h, W, T, ids = make(B, D, V, off)
    check_forward(h, W, T, ids, off, fs.token_logprobs(*dev(h, W, T, ids), vocab_offset=off))


@pytest.mark.parametrize("B,D,V", [s for s in SHAPES if s[1] % 32 == 0] + [(40, 96, 100), (200, 32, 530)])
@pytest.mark.parametrize("off", [0, 1, 1002, 7])
def test_forward_fragment_order(B, D, V, off):
    h, W, T, ids = make(B, D, V, off, seed=2)
    hd, Wd, Td, idd = dev(h, W, T, ids)
    Wp = fs.pack_weights(Wd, off)
    check_forward(h, W, T, ids, off, fs.token_logprobs(hd, Wp, Td, idd, vocab_offset=off, V=V))


@pytest.mark.parametrize("B,D,V", [s for s in SHAPES if s[0] * s[2] < 400000])
@pytest.mark.parametrize("off", [0, 1001])
def test_backward(B, D, V, off):
    h, W, T, ids = make(B, D, V, off, seed=3)
    check_backward(*backward_case(h, W, T, ids, off))


@pytest.mark.parametrize("D", [1024, 1056, 2048, 2080, 4096, 4128, 5120, 5152, 6144, 6176, 8192])
@pytest.mark.parametrize("B", [1, 16, 17, 32])
def test_forward_streams_every_row_length(B, D):
    """Each slice length of the streaming kernels, whole and ragged, both layouts."""
    h, W, T, ids = make(B, D, 333, 6, seed=18)
    hd, Wd, Td, idd = dev(h, W, T, ids)
    check_forward(h, W, T, ids, 6, fs.token_logprobs(hd, Wd, Td, idd, vocab_offset=6))
    Wp = fs.pack_weights(Wd, 6)
    check_forward(h, W, T, ids, 6, fs.token_logprobs(hd, Wp, Td, idd, vocab_offset=6, V=333))


# one shape per tile of the logits: 256 x 64, 256 x 128, 256 x 256, 128 x 128, 64 x 128, 64 x 64
@pytest.mark.parametrize("B,D,V", [(200, 64, 16032), (500, 72, 16001), (1000, 64, 16030),
                                   (3833, 96, 2161), (513, 136, 2001), (60, 32, 803)])
def test_every_tile(B, D, V):
    h, W, T, ids = make(B, D, V, 3, seed=20)
    hd, Wd, Td, idd = dev(h, W, T, ids)
    check_forward(h, W, T, ids, 3, fs.token_logprobs(hd, Wd, Td, idd, vocab_offset=3))
    if D % 32 == 0:
        Wp = fs.pack_weights(Wd, 3)
        check_forward(h, W, T, ids, 3, fs.token_logprobs(hd, Wp, Td, idd, vocab_offset=3, V=V))
    check_backward(*backward_case(h, W, T, ids, 3))


@pytest.mark.parametrize("B,V", [(64, 40000), (128, 50000), (128, 16032)])
def test_fragment_order_in_tiles_that_read_it_once(B, V):
    h, W, T, ids = make(B, 64, V, 2, seed=21)
    hd, Wd, Td, idd = dev(h, W, T, ids)
    Wp = fs.pack_weights(Wd, 2)
    check_forward(h, W, T, ids, 2, fs.token_logprobs(hd, Wp, Td, idd, vocab_offset=2, V=V))


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(seed):
    g = torch.Generator().manual_seed(500 + seed)
    size = lambda lo, hi: int(round(math.exp(math.log(lo) + float(torch.rand(1, generator=g)) * math.log(hi / lo))))
    B, D, V = size(1, 900), 8 * size(1, 160), size(1, 3000)
    off = size(1, 2000) if seed % 3 else 0
    h, W, T, ids = make(B, D, V, off, seed=seed, ignore=(0.0, 0.3, 0.8)[seed % 3])
    check_forward(h, W, T, ids, off, fs.token_logprobs(*dev(h, W, T, ids), vocab_offset=off))
    check_backward(*backward_case(h, W, T, ids, off))


@pytest.mark.parametrize("B,D,V", [(5, 64, 9), (300, 136, 700), (700, 264, 1), (513, 2056, 300)])
def test_backward_where_all_rows_share_a_token(B, D, V):
    h, W, T, ids = make(B, D, V, seed=19)
    ids[:] = V // 2
    check_backward(*backward_case(h, W, T, ids, 0))


def test_backward_splits_the_vocabulary_for_few_tokens():
    # several parts of the vocabulary per tile of grad_h
    h, W, T, ids = make(70, 264, 9000, seed=4)
    check_backward(*backward_case(h, W, T, ids, 0))


def test_backward_in_slices():
    """More tokens than one slice of the vocabulary holds dz for: 2^20 rows of
    8 elements would need 2 GiB for 1000 vocabulary rows.  Rows are copies of
    16 different ones, so the expected result is small work."""
    k, n, D, V = 16, 1 << 20, 8, 1000
    h, W, T, ids = make(k, D, V, seed=5, temp=False, ignore=0.0)
    lp, lse = (x.float() for x in ref.logprobs(h, W, T, ids, 0))
    g = torch.linspace(-1, 1, k) / n
    want = ref.logprobs_backward(h, W, T, ids, 0, lp, lse, g)
    rep = n // k
    hd, idd, lpd, lsed, gd = (x.cuda().repeat(rep, *[1] * (x.dim() - 1)) for x in (h, ids, lp, lse, g))
    gh, gw = fs.token_logprobs_backward(hd, W.cuda(), None, idd, lpd, lsed, gd)
    e = ref.logit_tolerance(h, W, T) + 2.0 ** -23 * float(lse.abs().max())
    assert torch.equal(gh.view(rep, k, D), gh[:k].expand(rep, k, D))
    check_backward((gh[:k], None), want, e)
    # sums of n equal terms in fp32, taken in steps of at least 8 products: 2^17
    # additions, each off by at most 2^-24 of a running sum that is half the
    # final one on average: 2^-8 relative
    w, bound = want[1] * rep, want[3] * rep
    tol = bound * (2.0 ** -8 + 2 * e + 2.0 ** -8) + 2.0 ** -8 * w.abs()
    assert ((gw.cpu().double() - w).abs() <= tol).all()


def test_one_gradient_alone():
    h, W, T, ids = make(50, 128, 400, seed=6)
    both, _, _ = backward_case(h, W, T, ids, 0)
    only_h, _, _ = backward_case(h, W, T, ids, 0, need_W=False)
    only_w, _, _ = backward_case(h, W, T, ids, 0, need_h=False)
    assert only_h[1] is None and only_w[0] is None
    assert torch.equal(only_h[0], both[0]) and torch.equal(only_w[1], both[1])


def test_rows_without_a_token_may_hold_anything():
    h, W, T, ids = make(70, 128, 300, seed=7)
    ids[::3] = -1
    bad = ids < 0
    lp, lse = (x.float() for x in ref.logprobs(h, W, T, ids, 0))
    g = torch.randn(70, generator=torch.Generator().manual_seed(1))
    want = ref.logprobs_backward(h, W, T, ids, 0, lp, lse, g)
    h2, T2, lp2, lse2, g2 = h.clone(), T.clone(), lp.clone(), lse.clone(), g.clone()
    for x in (h2, lp2, lse2, g2):
        x[bad] = math.nan
    h2[3], T2[bad] = math.inf, math.nan   # row 3 has no token
    got = fs.token_logprobs_backward(*dev(h2, W, T2, ids, lp2, lse2, g2))
    check_backward(got, want, ref.logit_tolerance(h, W, T) + 2.0 ** -23 * float(lse.abs().max()))
    assert (got[0][bad.cuda()] == 0).all()


@pytest.mark.parametrize("B", [1, 40, 300])
def test_no_row_has_a_token(B):
    h, W, T, ids = make(B, 64, 300, seed=8)
    ids[:] = -1
    z = torch.zeros(B)
    gh, gw = fs.token_logprobs_backward(*dev(h, W, T, ids, z, z, z + 1))
    assert not gh.any() and not gw.any()
    lp, lse = fs.token_logprobs(*dev(h, W, T, ids))
    assert not lp.any() and torch.isfinite(lse).all()


def test_no_rows():
    W = torch.randn(30, 16).to(torch.bfloat16).cuda()
    h, f, i = torch.empty(0, 16, dtype=torch.bfloat16).cuda(), torch.empty(0).cuda(), \
        torch.empty(0, dtype=torch.int32).cuda()
    lp, lse = fs.token_logprobs(h, W, None, i)
    assert lp.shape == (0,) and lse.shape == (0,)
    gw = torch.full((30, 16), 7.0, dtype=torch.bfloat16).cuda()
    fs.token_logprobs_backward(h, W, None, i, f, f, f, out=(None, gw))
    assert not gw.any()


@pytest.mark.parametrize("B", [2, 40, 300])
def test_nearly_certain_token(B):
    """The target far above the rest: log p ~ -exp(-gap) keeps its relative
    accuracy, and so does the gradient that carries 1 - p."""
    D, V = 64, 500
    g = torch.Generator().manual_seed(9)
    h = torch.ones(B, D).to(torch.bfloat16)
    W = (torch.randn(V, D, generator=g) * 0.02).to(torch.bfloat16)
    W[7] = 0.4   # logit 25.6 against ~0.16
    ids = torch.full((B,), 7, dtype=torch.int32)
    lp, lse = fs.token_logprobs(*dev(h, W, None, ids))
    want, _ = ref.logprobs(h, W, None, ids, 0)
    e = ref.logit_tolerance(h, W, None)
    assert float(want[0]) > -1e-7
    assert ((lp.cpu().double() / want - 1).abs() <= 2 * e + 2.0 ** -20).all()
    got, wantg, e = backward_case(h, W, None, ids, 0)
    check_backward(got, wantg, e)


def test_infinite_and_nan_inputs_stay_in_their_rows():
    h, W, T, ids = make(40, 64, 300, seed=10, temp=False, ignore=0.0)
    clean = fs.token_logprobs(*dev(h, W, T, ids))
    h[5, 3] = math.nan
    h[9, 0] = math.inf
    lp, lse = fs.token_logprobs(*dev(h, W, T, ids))
    assert lse[5].isnan() and lp[5].isnan() and not torch.isfinite(lse[9])
    keep = [b for b in range(40) if b not in (5, 9)]
    assert torch.equal(lp[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])


def test_infinite_temperature_is_uniform():
    h, W, _, ids = make(8, 64, 300, seed=11, temp=False, ignore=0.0)
    for B in (8, 40):
        hh, ii = h.repeat(5, 1)[:B], ids.repeat(5)[:B]
        lp, _ = fs.token_logprobs(*dev(hh, W, torch.full((B,), math.inf), ii))
        assert ((lp.cpu() + math.log(300)).abs() <= 2.0 ** -20 * math.log(300)).all()


def test_shards_add_up_to_the_whole():
    """Log-sum-exps merge, the owner's logprob + lse is the target's logit, and
    grad_h is the sum of the shards' shares."""
    B, D, V = 90, 192, 1000
    h, W, T, ids = make(B, D, V, seed=12)
    cuts = [0, 137, 600, 1000]
    hd, Wd, Td, idd = dev(h, W, T, ids)
    parts = [fs.token_logprobs(hd, Wd[a:b].contiguous(), Td, idd, vocab_offset=a)
             for a, b in zip(cuts, cuts[1:])]
    lse = torch.logsumexp(torch.stack([p[1] for p in parts]).double(), dim=0)
    logit = torch.stack([p[0] + p[1] for p in parts]).amax(dim=0).double()
    has = idd >= 0
    lp = torch.where(has, logit - lse, torch.zeros_like(lse))
    want_lp, want_lse = ref.logprobs(h, W, T, ids, 0)
    tol = 4 * ref.logit_tolerance(h, W, T) + 2.0 ** -20 * (1 + want_lse.abs())
    assert ((lse.cpu() - want_lse).abs() <= tol).all() and ((lp.cpu() - want_lp).abs() <= tol).all()
    g = torch.randn(B, generator=torch.Generator().manual_seed(2))
    lpf, lsef = want_lp.float(), want_lse.float()
    want = ref.logprobs_backward(h, W, T, ids, 0, lpf, lsef, g)
    e = ref.logit_tolerance(h, W, T) + 2.0 ** -23 * float(lsef.abs().max())
    share = []
    for a, b in zip(cuts, cuts[1:]):
        gh, gw = fs.token_logprobs_backward(hd, Wd[a:b].contiguous(), Td, idd, *dev(lpf, lsef, g),
                                            vocab_offset=a)
        tol = want[3][a:b] * (2.0 ** -8 + 2 * e + 2.0 ** -20) + 2.0 ** -8 * want[1][a:b].abs()
        assert ((gw.cpu().double() - want[1][a:b]).abs() <= tol).all()
        share.append(gh.double().cpu())
    total = sum(share)
    tol = want[2] * (2.0 ** -8 + 2 * e + 2.0 ** -20) + 2.0 ** -8 * sum(s.abs() for s in share)
    assert ((total - want[0]).abs() <= tol).all()


def test_gradient_against_differences_of_the_loss():
    """grad . direction equals the difference quotient of the fp64 loss."""
    B, D, V = 36, 64, 200
    h, W, T, ids = make(B, D, V, seed=13)
    (gh, gw), want, e = backward_case(h, W, T, ids, 0)
    g = torch.randn(B, generator=torch.Generator().manual_seed(1)) / B
    gen = torch.Generator().manual_seed(3)
    has = ids >= 0

    def loss(hh, WW):
        return float((ref.logprobs(hh, WW, T, ids, 0)[0] * g.double())[has].sum())
    for x, gx, bound, which in ((h, gh, want[2], 0), (W, gw, want[3], 1)):
        u = torch.randn(x.shape, generator=gen, dtype=torch.float64)
        eps = 1e-5
        d = ((loss(h.double() + eps * u, W.double()) - loss(h.double() - eps * u, W.double()))
             if which == 0 else
             (loss(h.double(), W.double() + eps * u) - loss(h.double(), W.double() - eps * u))) / (2 * eps)
        got = float((gx.cpu().double() * u).sum())
        tol = float((u.abs() * (bound * (2.0 ** -8 + 2 * e) + 2.0 ** -8 * gx.cpu().double().abs())).sum())
        assert abs(got - d) <= tol + 1e-8, (got, d, tol)


def test_equal_calls_give_equal_bits_and_outputs_can_be_given():
    h, W, T, ids = make(300, 256, 3000, seed=14)
    hd, Wd, Td, idd = dev(h, W, T, ids)
    a = fs.token_logprobs(hd, Wd, Td, idd)
    ws = torch.full((fs.token_logprobs_workspace_bytes(300, 256, 3000),), 255, dtype=torch.uint8).cuda()
    out = (torch.empty(300).cuda(), torch.empty(300).cuda())
    b = fs.token_logprobs(hd, Wd, Td, idd, out=out, workspace=ws)
    assert b[0] is out[0] and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    g = torch.randn(300).cuda()
    x = fs.token_logprobs_backward(hd, Wd, Td, idd, *a, g)
    ws = torch.full((fs.token_logprobs_backward_workspace_bytes(300, 256, 3000),), 255,
                    dtype=torch.uint8).cuda()
    y = fs.token_logprobs_backward(hd, Wd, Td, idd, *a, g, workspace=ws)
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.parametrize("B", [3, 40])
def test_head_beyond_32_bit_offsets(B):
    """W of 2.5e9 elements (4.9 GB): the rows past 2^31 elements are read, and
    their gradients written, where they are."""
    D, V = 8192, 300000
    g = torch.Generator(device="cuda").manual_seed(1)
    W = torch.empty(V, D, dtype=torch.bfloat16, device="cuda")
    for r in range(0, V, 50000):
        W[r:r + 50000] = torch.randn(50000, D, generator=g, device="cuda") * (1.5 / math.sqrt(D))
    h = torch.randn(B, D, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.tensor([V - 1, 7, V - 300] * B, dtype=torch.int32, device="cuda")[:B]
    lp, lse = fs.token_logprobs(h, W, None, ids)
    z = torch.cat([h.double() @ W[r:r + 50000].double().t() for r in range(0, V, 50000)], dim=1)
    # logits of size 1.5, |h . W| about 1.5: the tolerance of logit_tolerance, four deviations
    e = 4 * 2.0 ** -24 * math.sqrt(D) * 2.0 + 2.0 ** -23 * float(z.abs().max())
    want = torch.logsumexp(z, dim=1)
    zt = z.gather(1, ids.long()[:, None])[:, 0]
    assert ((lse.double() - want).abs() <= e + 2.0 ** -22 * want).all()
    assert ((lp.double() - (zt - want)).abs() <= 2 * e + 2.0 ** -21 * want).all()
    grad = torch.linspace(-1, 1, B, device="cuda")
    gh, gw = fs.token_logprobs_backward(h, W, None, ids, lp, lse, grad)
    dz = -torch.exp(z - lse.double()[:, None])
    dz[torch.arange(B), ids.long()] = -torch.expm1(lp.double())
    dz = dz * grad.double()[:, None]
    for rows in (slice(V - 400, V), slice(0, 50), slice(262100, 262200)):
        w = dz[:, rows].t() @ h.double()
        bound = dz[:, rows].abs().t() @ h.double().abs()
        tol = bound * (2.0 ** -8 + 4 * e + 2.0 ** -18) + 2.0 ** -8 * w.abs()
        assert ((gw[rows].double() - w).abs() <= tol).all()
    w, bound = torch.zeros_like(h, dtype=torch.float64), torch.zeros_like(h, dtype=torch.float64)
    for r in range(0, V, 50000):
        W64 = W[r:r + 50000].double()
        w += dz[:, r:r + 50000] @ W64
        bound += dz[:, r:r + 50000].abs() @ W64.abs()
    assert ((gh.double() - w).abs() <= bound * (2.0 ** -8 + 4 * e + 2.0 ** -18) + 2.0 ** -8 * w.abs()).all()


def test_two_streams_at_once():
    h, W, T, ids = make(70, 256, 3000, seed=15)
    hd, Wd, Td, idd = dev(h, W, T, ids)
    g = torch.randn(70).cuda()
    want = fs.token_logprobs(hd, Wd, Td, idd)
    wantg = fs.token_logprobs_backward(hd, Wd, Td, idd, *want, g)
    torch.cuda.synchronize()
    streams, res = [torch.cuda.Stream() for _ in range(2)], [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                r = fs.token_logprobs(hd, Wd, Td, idd)
                res[i] = (*r, *fs.token_logprobs_backward(hd, Wd, Td, idd, *r, g))
        torch.cuda.synchronize()
        for r in res:
            assert all(torch.equal(a, b) for a, b in zip(r, (*want, *wantg)))


@pytest.mark.parametrize("B,packed", [(1, True), (24, False), (90, False), (300, True)])
def test_captured_graph(B, packed):
    D, V = 256, 1500
    h, W, T, ids = make(B, D, V, seed=16)
    hd, Wd, Td, idd = dev(h, W, T, ids)
    Wf = fs.pack_weights(Wd) if packed else Wd
    g = torch.randn(B).cuda()
    ws = torch.empty(fs.token_logprobs_workspace_bytes(B, D, V), dtype=torch.uint8).cuda()
    wb = torch.empty(fs.token_logprobs_backward_workspace_bytes(B, D, V), dtype=torch.uint8).cuda()
    out = (torch.empty(B).cuda(), torch.empty(B).cuda())
    outg = (torch.empty_like(hd), torch.empty_like(Wd))

    def step():
        fs.token_logprobs(hd, Wf, Td, idd, out=out, workspace=ws, V=V)
        fs.token_logprobs_backward(hd, Wd, Td, idd, *out, g, out=outg, workspace=wb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        h2, _, _, ids2 = make(B, D, V, seed=20 + i)
        hd.copy_(h2)
        idd.copy_(ids2)
        wb.fill_(255 - i)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (*out, *outg)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (*out, *outg))), i


def test_refusals():
    h, W, T, ids = dev(*make(4, 64, 100, seed=17))
    with pytest.raises(ValueError):
        fs.token_logprobs(h, W[:, :32], T, ids)
    with pytest.raises(ValueError):
        fs.token_logprobs(h, W, T[:3], ids)
    with pytest.raises(TypeError):
        fs.token_logprobs(h, W, T, ids.long())
    with pytest.raises(ValueError):
        fs.token_logprobs(h, fs.pack_weights(W), T, ids)
    with pytest.raises(ValueError):
        fs.token_logprobs(h.t(), W, T, ids)
    with pytest.raises(fs.FlashSampleError):
        fs.token_logprobs(h, W, T, ids, workspace=torch.empty(64, dtype=torch.uint8).cuda())
    z = torch.zeros(4).cuda()
    with pytest.raises(ValueError):
        fs.token_logprobs(h, W, T, ids, out=(z, z))
    with pytest.raises(ValueError):
        fs.token_logprobs(h, W, T, ids, out=(T, z))
    with pytest.raises(ValueError):
        fs.token_logprobs(h, W, T, ids, workspace=W)
    with pytest.raises(ValueError):
        fs.token_logprobs_backward(h, W, T, ids, z, z, z, out=(h, None))
    with pytest.raises(ValueError):
        fs.token_logprobs_backward(h, W, T, ids, z, z, z, out=(None, W))
    with pytest.raises(fs.FlashSampleError):
        fs.token_logprobs_backward(h, W, T, ids, z, z, z, need_h=False, need_W=False)
    with pytest.raises(ValueError):
        fs.token_logprobs_backward(h, W, T, ids, z, z, z, out=(torch.empty_like(W), None))
