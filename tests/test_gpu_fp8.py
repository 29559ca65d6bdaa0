"""The LM head in 8-bit floating point against its plain reference (GPU).

Quantising: every byte.  Products: the dequantised tensors are exact in bf16, so
the references of the bf16 head apply to them.  Tolerances: a logit's fp32 sum of
exact products is off by at most training_ref.logit_tolerance; the 8-bit matrix
instructions, which more than 32 rows (16 with rows longer than 5120) take, add
fp8_ref.matrix_rounding; bf16 logits another 2^-8 of the value.  Log-probabilities
as in test_gpu_token_logprobs with that error of a logit."""
import math

import numpy as np
import pytest
import torch

import fp8_ref
import head_ref
import lm_head_exact_amd as fs
import parity
import training_ref as ref
from lm_head_exact_amd import workloads as wl

pytestmark = pytest.mark.gpu


def make(B, D, V, seed=0, scale=1.5, wide=True):
    g = torch.Generator().manual_seed(1000 * seed + B + D + V)
    h = torch.randn(B, D, generator=g)
    W = torch.randn(V, D, generator=g) * scale / math.sqrt(D)
    if wide:  # blocks of different sizes
        h = h * torch.exp(0.5 * torch.randn(B, 1, generator=g))
        W = W * torch.exp(0.3 * torch.randn(V, 1, generator=g))
    return h.to(torch.bfloat16), W.to(torch.bfloat16)


def u8(t):
    return t.contiguous().view(torch.uint8).cpu()


class Head:
    """A head, quantised by the library, and its reference."""

    def __init__(self, B, D, V, seed=0, **kw):
        self.h, self.W = make(B, D, V, seed, **kw)
        self.V, self.streams = V, (B <= 16 and D <= 8192) or (B <= 32 and D <= 5120)
        self.wq = fp8_ref.quantise(self.W, 128)
        self.hq = fp8_ref.quantise(self.h, 1)
        self.Wd = fp8_ref.dequantise(*self.wq, 128)
        self.hd = fp8_ref.dequantise(*self.hq, 1)
        q, s = fs.quantize_weights_fp8(self.W.cuda())
        assert torch.equal(u8(s), self.wq[1]) and torch.equal(u8(q), fp8_ref.pack(self.wq[0]))
        self.args = (self.h.cuda(), q, s, V)

    def logit_error(self, T=None, scores=False):
        """Largest error of a scaled logit, and of one of exact products (tokens are
        scored by those on up to 8192 entries)."""
        e = ref.logit_tolerance(self.hd, self.Wd, T)
        if self.streams or (scores and self.V <= 8192):
            return e, e
        m = fp8_ref.matrix_rounding(self.hq, self.wq) * ref.inv_temperature(T, self.h.shape[0])[:, None]
        return e + float(m.max()), e


SHAPES = [  # streaming kernels: every row length's, one and two tiles of 16 tokens
    (1, 64, 1), (3, 64, 17), (16, 192, 300), (2, 1024, 130), (5, 1088, 33), (7, 2112, 77), (4, 4096, 200),
    (3, 4160, 50), (6, 5120, 65), (2, 5184, 40), (9, 6208, 65), (16, 8192, 48), (17, 128, 515),
    (32, 1984, 130), (31, 4096, 99), (20, 5120, 100),
    # tiles; ragged in every direction
    (33, 64, 255), (64, 192, 257), (65, 128, 256), (128, 320, 511), (129, 320, 513), (257, 192, 1025),
    (20, 5184, 60), (17, 8192, 50), (33, 16384, 40)]
# one shape per tile: 256 x 64, 256 x 128, 256 x 256, 128 x 128, 64 x 64
TILES = [(200, 64, 16032), (500, 64, 16001), (1000, 64, 16030), (3833, 128, 2161), (513, 192, 2001),
         (60, 64, 803)]


@pytest.mark.parametrize("V,D", [(1, 64), (16, 128), (17, 192), (127, 320), (129, 64), (300, 576), (1000, 256)])
def test_quantised_weights(V, D):
    _, W = make(1, D, V, seed=1)
    codes, scales = fp8_ref.quantise(W, 128)
    q, s = fs.quantize_weights_fp8(W.cuda(), packed=False)
    assert q.shape == (V, D) and torch.equal(u8(q), codes) and torch.equal(u8(s), scales)
    p, s2 = fs.quantize_weights_fp8(W.cuda())
    assert torch.equal(u8(p), fp8_ref.pack(codes)) and torch.equal(u8(s2), scales)
    assert torch.equal(u8(fs.pack_weights_fp8(q)), u8(p))
    assert torch.equal(s.float().cpu(), torch.pow(2.0, scales.float() - 127))


@pytest.mark.parametrize("D", [8, 24, 136, 1000])
def test_row_major_takes_any_multiple_of_8(D):
    _, W = make(1, D, 150, seed=2)
    codes, scales = fp8_ref.quantise(W, 128)
    q, s = fs.quantize_weights_fp8(W.cuda(), packed=False)
    assert torch.equal(u8(q), codes) and torch.equal(u8(s), scales)


def test_every_value():
    """Every bf16 bit pattern, in blocks of one binade and in mixed ones."""
    x = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    for W in (x.view(512, 128), x.view(128, 512), x[torch.randperm(1 << 16, generator=torch.Generator().manual_seed(1))].view(256, 256)):
        W = W.contiguous()
        codes, scales = fp8_ref.quantise(W, 128)
        q, s = fs.quantize_weights_fp8(W.cuda(), packed=False)
        assert torch.equal(u8(s), scales)
        nan = codes & 0x7F == 0x7F
        got = u8(q)
        assert torch.equal(got[~nan], codes[~nan]) and ((got[nan] & 0x7F) == 0x7F).all()


@pytest.mark.parametrize("B,D,V", SHAPES)
def test_logits(B, D, V):
    c = Head(B, D, V)
    want = ref.scaled_logits(c.hd, c.Wd, None)
    e, _ = c.logit_error()
    z = fs.logits_fp8(*c.args).cpu().double()
    assert ((z - want).abs() <= e).all(), float((z - want).abs().max())
    b = fs.logits_fp8(*c.args, dtype=torch.bfloat16).cpu().double()
    assert ((b - want).abs() <= e + 2.0 ** -8 * (want.abs() + e)).all()
    # rows further apart than V, misaligned; what lies between them stays
    for pitch, at in ((V + 5, 0), (V + 3, 1), ((V + 15) // 8 * 8, 0)):
        for dt, full in ((torch.float32, z), (torch.bfloat16, b)):
            buf = torch.full((B * pitch + 8,), 7.0, dtype=dt, device="cuda")
            out = buf[at:at + B * pitch].view(B, pitch)[:, :V]
            assert fs.logits_fp8(*c.args, out=out) is out
            assert torch.equal(out.cpu().double(), full)
            rest = buf.clone()
            rest[at:at + B * pitch].view(B, pitch)[:, :V] = 7.0
            assert (rest == 7.0).all()


def check_scores(c, T, ids, off, got):
    lp, lse = (x.cpu().double() for x in got)
    want_lp, want_lse = ref.logprobs(c.hd, c.Wd, T, ids, off)
    e, exact = c.logit_error(T, scores=True)
    assert ((lse - want_lse).abs() <= e + 2.0 ** -22 * (1 + want_lse.abs())).all()
    fin = torch.isfinite(want_lp)
    assert torch.equal(torch.isinf(lp) & (lp < 0), ~fin)
    tol = (e + exact + 2.0 ** -22 * (1 + want_lp.abs())) * torch.clamp(want_lp.abs(), max=1.0)
    tol = tol + 2.0 ** -23 * want_lp.abs()
    assert ((lp - want_lp).abs()[fin] <= tol[fin]).all(), float(((lp - want_lp).abs() - tol)[fin].max())
    assert (lp[ids < 0] == 0).all()


def targets(B, V, off, seed=0):
    g = torch.Generator().manual_seed(seed + B)
    T = 0.4 + torch.rand(B, generator=g)
    T[3::5] = torch.tensor([0.0, -1.0, math.nan, 0.0])[torch.arange(len(T[3::5])) % 4]
    ids = torch.randint(0, V, (B,), generator=g) + off
    if off:
        ids[1::4] = torch.randint(0, off, (len(ids[1::4]),), generator=g)
        ids[2::7] = off + V + 5
    ids[0] = off + V - 1
    ids = torch.where(torch.rand(B, generator=g) < 0.2, torch.full_like(ids, -100), ids)
    return T, ids.to(torch.int32)


@pytest.mark.parametrize("B,D,V", SHAPES)
@pytest.mark.parametrize("off", [0, 1001])
def test_token_logprobs(B, D, V, off):
    c = Head(B, D, V, seed=3)
    T, ids = targets(B, V, off)
    check_scores(c, T, ids, off, fs.token_logprobs_fp8(*c.args, T.cuda(), ids.cuda(), vocab_offset=off))
    if off == 0:
        check_scores(c, None, ids, 0, fs.token_logprobs_fp8(*c.args, None, ids.cuda()))


@pytest.mark.parametrize("B,D,V", SHAPES)
@pytest.mark.parametrize("off", [0, 1004])
def test_samples(B, D, V, off):
    c = Head(B, D, V, seed=4)
    T, _ = targets(B, V, off)
    ids, val = fs.sample_fp8(*c.args, T.cuda(), 2 ** 40 + 7, 2 ** 33 + 5, vocab_offset=off)
    parity.check_rows(wl.bf16_bits(c.hd), wl.bf16_bits(c.Wd), T.numpy(), 2 ** 40 + 7, 2 ** 33 + 5, off,
                      ids.cpu().numpy(), val.cpu().numpy())

# and for tokens' scores, by exact products (up to 8192 entries) and by the 8-bit ones
SCORE_TILES = [(3000, 128, 700), (513, 64, 8192), (4000, 192, 2161), (3833, 128, 2161), (40, 128, 700),
               (200, 128, 8193), (513, 64, 8193), (1000, 64, 8193), (40, 192, 8193), (648, 192, 10821)]


@pytest.mark.parametrize("B,D,V", SCORE_TILES)
def test_scores_by_every_tile(B, D, V):
    """At temperatures down to 0.1, where few entries carry the log-sum-exp."""
    c = Head(B, D, V, seed=12, wide=False)
    T, ids = targets(B, V, 0)
    T[1::3] = 0.1
    check_scores(c, T, ids, 0, fs.token_logprobs_fp8(*c.args, T.cuda(), ids.cuda()))


@pytest.mark.parametrize("B,D,V", TILES)
def test_every_tile(B, D, V):
    c = Head(B, D, V, seed=5, wide=False)
    want = ref.scaled_logits(c.hd, c.Wd, None)
    e, _ = c.logit_error()
    z = fs.logits_fp8(*c.args).cpu().double()
    assert ((z - want).abs() <= e).all()
    b = fs.logits_fp8(*c.args, dtype=torch.bfloat16).cpu().double()
    assert ((b - want).abs() <= e + 2.0 ** -8 * (want.abs() + e)).all()
    T, ids = targets(B, V, 8)
    check_scores(c, T, ids, 8, fs.token_logprobs_fp8(*c.args, T.cuda(), ids.cuda(), vocab_offset=8))
    i, v = fs.sample_fp8(*c.args, T.cuda(), 3, 4, vocab_offset=8)
    rows = np.unique(np.linspace(0, B - 1, 40).astype(np.int32))
    parity.check_rows(wl.bf16_bits(c.hd), wl.bf16_bits(c.Wd), T.numpy(), 3, 4, 8, i.cpu().numpy(),
                      v.cpu().numpy(), rows=rows)


def test_a_row_in_any_batch():
    """One row's logits alone and among 32 are the same sums of exact products."""
    c = Head(32, 4096, 400, seed=6)
    z = fs.logits_fp8(*c.args)
    alone = fs.logits_fp8(c.args[0][7:8], *c.args[1:])
    e, _ = c.logit_error()
    assert ((z[7:8] - alone).abs() <= 2 * e).all()


@pytest.mark.parametrize("B", [5, 40])
def test_not_finite(B):
    """NaN and infinities of h or W stay in the logits that they enter."""
    h, W = make(B, 192, 300, seed=7)
    h[1, 3], h[2, 150], W[7, 0], W[130, 191] = math.nan, math.inf, math.nan, -math.inf
    q, s = fs.quantize_weights_fp8(W.cuda())
    z = fs.logits_fp8(h.cuda(), q, s, 300).cpu()
    bad = torch.zeros(B, 300, dtype=torch.bool)
    bad[1], bad[2], bad[:, 7], bad[:, 130] = True, True, True, True
    assert torch.equal(torch.isnan(z), bad) and torch.isfinite(z[~bad]).all()
    ok = fs.quantize_weights_fp8(torch.where(torch.isfinite(W), W, torch.zeros_like(W)).cuda())
    lp, lse = fs.token_logprobs_fp8(h.cuda(), *ok, 300, None, torch.full((B,), 5, dtype=torch.int32).cuda())
    nan = torch.zeros(B, dtype=torch.bool)
    nan[1:3] = True
    assert torch.equal(torch.isnan(lp).cpu(), nan) and torch.equal(torch.isnan(lse).cpu(), nan)


@pytest.mark.parametrize("B", [3, 40])
@pytest.mark.parametrize("size", [1e-30, 1e30])
def test_far_scales(B, size):
    """Blocks far from 1: the scales carry them."""
    h, W = make(B, 128, 200, seed=8)
    h, W = (h.float() * size).to(torch.bfloat16), (W.float() / size).to(torch.bfloat16)
    q, s = fs.quantize_weights_fp8(W.cuda())
    hq, wq = fp8_ref.quantise(h, 1), fp8_ref.quantise(W, 128)
    want = ref.scaled_logits(fp8_ref.dequantise(*hq, 1), fp8_ref.dequantise(*wq, 128), None)
    e = ref.logit_tolerance(fp8_ref.dequantise(*hq, 1), fp8_ref.dequantise(*wq, 128), None)
    if B > 32:
        e += float(fp8_ref.matrix_rounding(hq, wq).max())
    assert ((fs.logits_fp8(h.cuda(), q, s, 200).cpu().double() - want).abs() <= e).all()


def test_no_rows_and_zeros():
    c = Head(4, 128, 100, seed=9)
    h0 = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    assert fs.logits_fp8(h0, *c.args[1:]).shape == (0, 100)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert fs.token_logprobs_fp8(h0, *c.args[1:], None, none)[0].shape == (0,)
    assert fs.sample_fp8(h0, *c.args[1:], torch.empty(0, device="cuda"), 1, 2)[0].shape == (0,)
    assert (fs.logits_fp8(torch.zeros_like(c.args[0]), *c.args[1:]) == 0).all()


@pytest.mark.parametrize("B", [8, 100])
def test_shards_merge(B):
    """Samples of four shards, merged, against the whole head."""
    c = Head(B, 128, 1024, seed=10)
    T, _ = targets(B, 1024, 0)
    T = T.cuda()
    pv, pi = torch.empty(4, B, device="cuda"), torch.empty(4, B, dtype=torch.int32, device="cuda")
    for r in range(4):
        q, s = fs.quantize_weights_fp8(c.W[256 * r:256 * r + 256].cuda())
        pi[r], pv[r] = fs.sample_fp8(c.args[0], q, s, 256, T, 9, 1, vocab_offset=256 * r)
    ids, val = fs.merge(pv, pi)
    parity.check_rows(wl.bf16_bits(c.hd), wl.bf16_bits(c.Wd), T.cpu().numpy(), 9, 1, 0, ids.cpu().numpy(),
                      val.cpu().numpy())


@pytest.mark.parametrize("B", [20, 90])
def test_given_outputs_and_refusals(B):
    c = Head(B, 256, 500, seed=11)
    h, q, s, V = c.args
    T, ids = (x.cuda() for x in targets(B, V, 0))
    n = fs.fp8_workspace_bytes(B, 256, V)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    lp, lse = torch.full((B,), 7.0, device="cuda"), torch.full((B,), 7.0, device="cuda")
    want = fs.token_logprobs_fp8(*c.args, T, ids)
    got = fs.token_logprobs_fp8(*c.args, T, ids, out=(lp, lse), workspace=ws)
    assert got[0] is lp and torch.equal(lp, want[0]) and torch.equal(lse, want[1])
    si, sv = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, device="cuda")
    want = fs.sample_fp8(*c.args, T, 5, 6)
    before = sv._version
    fs.sample_fp8(*c.args, T, 5, 6, out=(si, sv), workspace=ws)
    assert torch.equal(si, want[0]) and torch.equal(sv, want[1]) and sv._version > before
    for call in (lambda **k: fs.token_logprobs_fp8(*c.args, T, ids, **k),
                 lambda **k: fs.sample_fp8(*c.args, T, 5, 6, **k), lambda **k: fs.logits_fp8(*c.args, **k)):
        with pytest.raises(fs.FlashSampleError):
            call(workspace=ws[:n - 256])
        with pytest.raises(ValueError, match="overlap"):
            call(workspace=h.view(-1).view(torch.uint8))
    with pytest.raises(ValueError, match="overlap"):
        fs.sample_fp8(*c.args, T, 5, 6, out=(si, T))
    with pytest.raises(ValueError, match="overlap"):
        fs.quantize_weights_fp8(c.W.cuda(), out=(q, q[:8].view(torch.float8_e8m0fnu).view(4, 2)))
    with pytest.raises(ValueError, match="fragment order"):
        fs.logits_fp8(h, fs.quantize_weights_fp8(c.W.cuda(), packed=False)[0], s, V)
    for bad in ((h, q, s, V + 16), (h, q[:-1024], s, V), (h, q, s[:-1], V), (h[:, :192], q, s, V)):
        with pytest.raises(ValueError):
            fs.logits_fp8(*bad)
    with pytest.raises(TypeError):
        fs.logits_fp8(h, q.view(torch.uint8), s, V)
    with pytest.raises(TypeError):
        fs.logits_fp8(*c.args, dtype=torch.float16)
    wide = torch.empty(B, 2 * V, device="cuda")
    for out in (wide[:, ::2], wide[:, :V].t().contiguous().t(), wide[:1, :V].expand(B, V)):
        with pytest.raises(ValueError):
            fs.logits_fp8(*c.args, out=out)
    with pytest.raises(fs.FlashSampleError):
        fs.sample_fp8(*c.args, T, 5, 6, vocab_offset=2)
    with pytest.raises(fs.FlashSampleError):
        fs.quantize_weights_fp8(c.W[:, :200].contiguous().cuda())
    with pytest.raises(ValueError, match="2\\^31"):
        fs.token_logprobs_fp8(*c.args, T, ids, vocab_offset=2 ** 32)


@pytest.mark.parametrize("B", [4, 40])
def test_no_gradient_leads_through(B):
    """Results of an h that requires a gradient equal the others; their backward pass
    raises.  Nothing is recorded without gradients or into given outputs."""
    c = Head(B, 128, 200, seed=13)
    h = c.args[0].clone().requires_grad_(True)
    _, ids = targets(B, 200, 0)
    ids = ids.cuda()
    z, want = fs.logits_fp8(h, *c.args[1:]), fs.logits_fp8(*c.args)
    lp, lse = fs.token_logprobs_fp8(h, *c.args[1:], None, ids)
    wlp, wlse = fs.token_logprobs_fp8(*c.args, None, ids)
    assert torch.equal(z, want) and torch.equal(lp, wlp) and torch.equal(lse, wlse)
    for y in (z, lp, lse):
        with pytest.raises(RuntimeError, match="8-bit head"):
            y.sum().backward()
    assert h.grad is None
    with torch.no_grad():
        assert not fs.logits_fp8(h, *c.args[1:]).requires_grad
    assert not fs.logits_fp8(h, *c.args[1:], out=torch.empty_like(want)).requires_grad
    assert not fs.sample_fp8(h, *c.args[1:], torch.ones(B, device="cuda"), 1, 2)[1].requires_grad


@pytest.mark.parametrize("B", [12, 70])
def test_graph_replays(B):
    """Quantising, sampling, scoring and logits in one graph, replayed on new weights."""
    c = Head(B, 256, 900, seed=12)
    h, W = c.h.cuda(), c.W.cuda()
    T, _ = (x.cuda() for x in targets(B, 900, 0))
    q, s = (torch.empty_like(x) for x in c.args[1:3])
    n = fs.fp8_workspace_bytes(B, 256, 900)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    ids, val = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, device="cuda")
    lp, lse, z = torch.empty(B, device="cuda"), torch.empty(B, device="cuda"), torch.empty(B, 900, device="cuda")

    def steps():
        fs.quantize_weights_fp8(W, out=(q, s))
        fs.sample_fp8(h, q, s, 900, T, 3, 1, out=(ids, val), workspace=ws)
        fs.token_logprobs_fp8(h, q, s, 900, T, ids, out=(lp, lse), workspace=ws)
        fs.logits_fp8(h, q, s, 900, out=z, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        steps()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        steps()
    for i in range(4):
        nh, nw = make(B, 256, 900, seed=20 + i)
        h.copy_(nh)
        W.copy_(nw)
        g.replay()
        torch.cuda.synchronize()
        wq, wsc = fs.quantize_weights_fp8(W)
        wi, wv = fs.sample_fp8(h, wq, wsc, 900, T, 3, 1)
        wl_, ws_ = fs.token_logprobs_fp8(h, wq, wsc, 900, T, wi)
        wz = fs.logits_fp8(h, wq, wsc, 900)
        for a, b in ((u8(q), u8(wq)), (u8(s), u8(wsc)), (ids, wi), (val, wv), (lp, wl_), (lse, ws_), (z, wz)):
            assert torch.equal(a, b), i


def test_two_streams_at_once():
    cs = [Head(B, 512, 3000, seed=30 + B) for B in (24, 80)]
    want = [fs.logits_fp8(*c.args) for c in cs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cs], []
    for st, c in zip(streams, cs):
        with torch.cuda.stream(st):
            got.append([fs.logits_fp8(*c.args) for _ in range(6)])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(x, w) for x in g)


def test_logits_past_2_31_elements():
    """Rows of the logits beyond 2^31 elements (fp32, 9.7 GB)."""
    B, D, V = 20000, 64, 121000
    g = torch.Generator(device="cuda").manual_seed(3)
    h = torch.randn(B, D, generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn(V, D, generator=g, device="cuda") / 8).to(torch.bfloat16)
    q, s = fs.quantize_weights_fp8(W)
    z = fs.logits_fp8(h, q, s, V)
    for rows in (slice(0, 40), slice(17740, 17790), slice(19960, 20000)):   # around 2^31 and the end
        assert torch.equal(z[rows], fs.logits_fp8(h[rows].contiguous(), q, s, V))


def test_the_rollout_of_a_training_step():
    """Train the head, quantise it, sample and score with it: cross entropy, an update
    of the weights, 8-bit weights, samples, their log-probabilities and logits."""
    B, D, V = 60, 128, 700
    h, W = (x.cuda() for x in make(B, D, V, seed=40, wide=False))
    t = torch.randint(0, V, (B,), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    for _ in range(3):
        _, _, gh, gw = fs.cross_entropy(h, W, t, z_loss=1e-4)
        want = head_ref.cross_entropy(h, W, t, z_loss=1e-4)
        assert (gw.double() - want["grad_W"]).norm() <= 2.0 ** -7 * want["grad_W"].norm()
        fs.clip_grad_norm([gw, gh], 1.0)
        W = (W.float() - 2.0 * gw.float()).to(torch.bfloat16)
    q, s = fs.quantize_weights_fp8(W)
    T = torch.full((B,), 0.9, device="cuda")
    ids, _ = fs.sample_fp8(h, q, s, V, T, 8, 0)
    lp, lse = fs.token_logprobs_fp8(h, q, s, V, T, ids)
    z = fs.logits_fp8(h, q, s, V).double() / 0.9
    want = torch.log_softmax(z, dim=1).gather(1, ids.long()[:, None])[:, 0]
    assert (lp.double() - want).abs().max() <= 1e-3 and (lse.double() - torch.logsumexp(z, 1)).abs().max() <= 1e-3
    # the quantised policy near the one in training: e4m3 is off by 2^-4 of a value at
    # most, so a logit by 2^-3 of the sum of its products' sizes
    bf, _ = fs.token_logprobs(h, W, T, ids)
    size = (h.double().abs() @ W.double().abs().t()).max() / 0.9
    assert (lp - bf).abs().max() <= 2 * (2.0 ** -3 + 2.0 ** -8) * float(size)
