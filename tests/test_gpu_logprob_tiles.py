"""Token log-probabilities and their gradient by every tile of their products,
against fp64, the gradient in norm as well as by element (GPU).  The logits'
tiles that the cases name are checked against the library's rule by
test_tile_rule.py.

Tolerance in norm.  Rounding to bf16 (8 significant bits) is off by a uniform
error of up to half a step: root mean square 2^-8 / sqrt(3) relative to a value
of mantissa 1, over mantissas of uniform logarithm sqrt(3 / (8 ln 2)) of that,
RHO = 1.66e-3.  A gradient x = sum of dz w is rounded once (RHO |x|), and so is
every dz but the target's, independently (RHO sqrt(sum dz^2 w^2)).  Both norms
are over at least 2500 elements, so that the actual one stays within a tenth of
the expected; logits off by e, and sums in fp32, add (2 e + 2^-20) sum |dz| |w|."""
import math

import pytest
import torch

import lm_head_exact_amd as fs
import training_ref as ref
from test_gpu_token_logprobs import backward_case, check_backward, check_forward, dev, make

pytestmark = pytest.mark.gpu
RHO = 2.0 ** -8 / math.sqrt(3) * math.sqrt(3 / (8 * math.log(2)))

# rows, row length, vocabulary, and the tile of the logits: vocabulary rows x tokens
CASES = [
    (60, 136, 803, (64, 64)), (300, 64, 701, (64, 64)),
    (300, 264, 5000, (64, 128)), (100, 136, 9001, (64, 128)), (800, 72, 2003, (64, 128)),
    (3833, 96, 2161, (128, 128)),
    (200, 72, 16032, (256, 64)),
    (500, 64, 16001, (256, 128)),
    (1000, 72, 16030, (256, 256)), (820, 128, 16001, (256, 256)),
]

# the same for the forward call, more tokens than one tile's and not (W in
# fragment order is then read past the caches)
FORWARD = [
    (100, 96, 2001, (64, 64)), (60, 64, 2001, (64, 64)), (300, 96, 5000, (64, 128)),
    (100, 160, 9001, (64, 128)), (3833, 96, 2161, (128, 128)), (300, 96, 9001, (256, 64)),
    (64, 96, 40000, (256, 64)), (500, 96, 9001, (256, 128)), (128, 32, 40000, (256, 128)),
    (800, 96, 12000, (256, 256)), (200, 32, 40000, (256, 256)),
]
name = lambda x: "x".join(map(str, x)) if isinstance(x, tuple) else str(x)


@pytest.mark.parametrize("B,D,V,tile", FORWARD, ids=name)
@pytest.mark.parametrize("off", [0, 1003])
def test_log_probabilities_by_every_tile(B, D, V, tile, off):
    h, W, T, ids = make(B, D, V, off, seed=40)
    hd, Wd, Td, idd = dev(h, W, T, ids)
    check_forward(h, W, T, ids, off, fs.token_logprobs(hd, Wd, Td, idd, vocab_offset=off))
    Wp = fs.pack_weights(Wd, off)
    check_forward(h, W, T, ids, off, fs.token_logprobs(hd, Wp, Td, idd, vocab_offset=off, V=V))


def check_norms(got, want, dz, h, W, e):
    """dz in fp64, without the targets' own terms."""
    for x, w, bound, spread in ((got[0], want[0], want[2], (dz ** 2) @ (W ** 2)),
                                (got[1], want[1], want[3], (dz ** 2).T @ (h ** 2))):
        tol = (1.1 * RHO * math.sqrt(float((w ** 2).sum() + spread.sum()))
               + (2 * e + 2.0 ** -20) * float(bound.norm()))
        err = float((x.to(w) - w).norm())
        assert err <= tol, (err, tol, err / float(w.norm()))


def other_rows(h, W, T, ids, off, lse, grad):
    """dz of the rows that are no token's own, and h with zeros in rows without a token."""
    t = ref.scaled_logits(h, W, T)
    dz = -torch.exp(t - lse.double()[:, None]) * (grad.double() * ref.inv_temperature(T, len(ids)))[:, None]
    for b, i in enumerate(ids.tolist()):
        if i < 0:
            dz[b] = 0
        elif off <= i < off + W.shape[0]:
            dz[b, i - off] = 0
    return dz, torch.where((ids >= 0)[:, None], h.double(), torch.zeros((), dtype=torch.float64))


@pytest.mark.parametrize("B,D,V,tile", CASES, ids=name)
@pytest.mark.parametrize("off", [0, 1001])
def test_gradient_by_every_tile(B, D, V, tile, off):
    h, W, T, ids = make(B, D, V, off, seed=41)
    got, want, e = backward_case(h, W, T, ids, off)
    check_backward(got, want, e)
    grad = torch.randn(B, generator=torch.Generator().manual_seed(1)) / B   # (backward_case's)
    lse = ref.logprobs(h, W, T, ids, off)[1].float()
    dz, hz = other_rows(h, W, T, ids, off, lse, grad)
    check_norms([x.cpu() for x in got], want, dz, hz, W.double(), e)


@pytest.mark.parametrize("B", [520, 1300])
def test_gradient_of_a_long_head(B):
    """Vocabularies and rows so long that the gradient of W goes by tiles of 256 x
    256, against fp64 on the device."""
    D, V = 8192, 32600
    g = torch.Generator(device="cuda").manual_seed(B)
    W = (torch.randn(V, D, generator=g, device="cuda") * (1.5 / math.sqrt(D))).to(torch.bfloat16)
    h = torch.randn(B, D, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.randint(0, V, (B,), generator=g, device="cuda").to(torch.int32)
    ids[::6] = -1
    ids[5:9] = 77
    grad = torch.randn(B, generator=g, device="cuda") / B
    h64, W64, has = h.double(), W.double(), ids >= 0
    z = h64 @ W64.t()
    lse = torch.logsumexp(z, dim=1).float()
    lp = torch.where(has, z.gather(1, ids.clamp(min=0).long()[:, None])[:, 0] - lse.double(),
                     torch.zeros_like(lse, dtype=torch.float64)).float()
    gh, gw = fs.token_logprobs_backward(h, W, None, ids, lp, lse, grad)
    # logits of size 1.5 and |h . W| about 1.5: logit_tolerance's, four deviations
    e = 4 * 2.0 ** -24 * math.sqrt(D) * 2.0 + 2.0 ** -23 * float(z.abs().max() + lse.max())
    dz = torch.where(has[:, None], -torch.exp(z - lse.double()[:, None]) * grad.double()[:, None],
                     torch.zeros((), dtype=torch.float64, device="cuda"))
    del z
    rows = torch.arange(B, device="cuda")[has]
    others = dz.clone()
    others[rows, ids[has].long()] = 0
    dz[rows, ids[has].long()] = (-torch.expm1(lp.double()) * grad.double())[has]
    want = [dz @ W64, dz.t() @ h64, dz.abs() @ W64.abs(), dz.abs().t() @ h64.abs()]
    for x, w, bound in ((gh, want[0], want[2]), (gw, want[1], want[3])):
        tol = bound * (2.0 ** -8 + 2 * e + 2.0 ** -20) + 2.0 ** -8 * w.abs()
        assert ((x.double() - w).abs() <= tol).all()
    check_norms((gh, gw), want, others, torch.where(has[:, None], h64, torch.zeros_like(h64)), W64, e)
