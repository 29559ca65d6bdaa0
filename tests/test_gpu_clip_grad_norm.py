"""fs_clip_grad_norm against plain fp64 (GPU).

Tolerances.  Squares and their sum are fp64, the norm is rounded once to
fp32 (2^-24).  The factor is rounded to fp32 (2^-24), so is its product with
an element (2^-24), and the result to its type (half a step: bf16 2^-8, fp16
2^-11, and for fp16 half its smallest step, 2^-25)."""
import math

import pytest
import torch

import lm_head_exact_amd as fs
import training_ref as ref

pytestmark = pytest.mark.gpu
HALF = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}


def tensors(sizes, dtypes, seed=0, rms=0.01):
    g = torch.Generator().manual_seed(seed + len(sizes))
    return [(rms * torch.randn(n, generator=g)).to(dtypes[i % len(dtypes)]) for i, n in enumerate(sizes)]


def check(grads, max_norm, in_place):
    want_norm, want = ref.clip(grads, max_norm)
    dev = [g.cuda() for g in grads]
    out = None if in_place else [torch.full_like(g, 5.0) for g in dev]
    norm = fs.clip_grad_norm(dev, max_norm, out=out)
    assert abs(float(norm) - want_norm) <= 2.0 ** -23 * want_norm
    for g, d, w in zip(grads, dev if in_place else out, want):
        tol = w.abs() * (HALF[g.dtype] + 3 * 2.0 ** -24) + TINY[g.dtype]
        assert ((d.cpu().double() - w).abs() <= tol).all()
    if not in_place:
        assert all(torch.equal(g, d.cpu()) for g, d in zip(grads, dev))


SIZES = [[1], [7], [0, 3, 0], [4096, 4097, 1, 255, 256, 257], [32768, 32769, 65537, 16385],
         [200000, 5], [13] * 95, [13] * 96, [13] * 97, [200] * 300, [1 << 21]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("in_place", [True, False])
def test_clip(sizes, dtype, in_place):
    grads = tensors(sizes, [dtype])
    norm = ref.clip(grads, 1.0)[0]
    check(grads, 0.3 * norm, in_place)      # scaled
    check(grads, 3.0 * norm + 1.0, in_place)  # left alone


def test_mixed_types_shapes_and_odd_addresses():
    base = tensors([100003], [torch.float32])[0]
    grads = [base[1:5000].view(torch.float32).clone(), tensors([3 * 5 * 7], [torch.float16])[0].view(3, 5, 7),
             tensors([70001], [torch.bfloat16])[0]]
    check(grads, 0.01, True)
    dev = base.cuda()
    b16 = base.to(torch.bfloat16).cuda()
    views = [dev[1:40002], dev[50001:100000], b16[3:99998]]   # 4- and 2-byte aligned
    want_norm, want = ref.clip(views, 0.02)
    norm = fs.clip_grad_norm(views, 0.02)
    assert abs(float(norm) - want_norm) <= 2.0 ** -23 * want_norm
    for v, w in zip(views, want):
        tol = w.abs() * (HALF[v.dtype] + 3 * 2.0 ** -24) + TINY[v.dtype]
        assert ((v.cpu().double() - w).abs() <= tol).all()
    # what lies beside the views is untouched
    assert dev[0] == base[0] and torch.equal(dev[40002:50001].cpu(), base[40002:50001])
    assert torch.equal(b16[:3].cpu(), base[:3].to(torch.bfloat16))


@pytest.mark.parametrize("value", [1e30, 1e-30])
def test_squares_beyond_fp32(value):
    """fp64 squares: gradients whose squares leave fp32's range have a norm."""
    grads = [torch.full((3000,), value), torch.full((5,), -value)]
    want = value * math.sqrt(3005)
    dev = [g.cuda() for g in grads]
    norm = fs.clip_grad_norm(dev, math.inf)
    assert abs(float(norm) / want - 1) <= 2.0 ** -22
    assert all(torch.equal(g, d.cpu()) for g, d in zip(grads, dev))
    fs.clip_grad_norm(dev, 1.0)
    if value > 1:
        assert abs(float(dev[0][0]) / (1 / math.sqrt(3005)) - 1) <= 2.0 ** -21


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_norm_that_is_not_finite_scales_nothing(bad):
    grads = tensors([5000, 70000], [torch.bfloat16, torch.float32])
    grads[1][69999] = bad
    dev = [g.cuda() for g in grads]
    out = [torch.zeros_like(g) for g in dev]
    norm = fs.clip_grad_norm(dev, 1e-3, out=out)
    assert not torch.isfinite(norm).any()
    for g, o in zip(grads, out):
        assert torch.equal(torch.nan_to_num(g.float(), nan=7.0), torch.nan_to_num(o.cpu().float(), nan=7.0))
    fs.clip_grad_norm(dev, 1e-3)
    assert torch.equal(dev[0].cpu(), grads[0])


def test_more_elements_than_32_bits_count():
    n = (1 << 31) + 12345
    x = torch.full((n,), 2.0 ** -10, dtype=torch.bfloat16, device="cuda")
    x[-1] = 1.0
    want = math.sqrt((n - 1) * 2.0 ** -20 + 1.0)
    norm = fs.clip_grad_norm([x], want / 2)
    assert abs(float(norm) / want - 1) <= 2.0 ** -23
    # times 1/2 exactly but for the 1e-6 in the divisor: below half a step
    assert float(x[-1]) == 0.5 and float(x[n // 2]) == 2.0 ** -11 and float(x[(1 << 31) - 1]) == 2.0 ** -11


def test_zero_gradients_and_zero_limit():
    z = [torch.zeros(1000).cuda()]
    assert float(fs.clip_grad_norm(z, 1.0)) == 0.0 and not z[0].any()
    x = [torch.ones(1000).cuda()]
    fs.clip_grad_norm(x, 0.0)
    assert not x[0].any()


def test_equal_calls_give_equal_bits_and_a_captured_graph_replays():
    grads = [g.cuda() for g in tensors([70001, 300000, 12], [torch.bfloat16, torch.float32])]
    out = [torch.empty_like(g) for g in grads]
    norm = torch.empty(1).cuda()
    import ctypes
    from lm_head_exact_amd import binding as bd
    sizes = (ctypes.c_int64 * 3)(*[g.numel() for g in grads])
    ws = torch.empty(bd.lib().fs_clip_grad_norm_workspace_bytes(sizes, 3), dtype=torch.uint8).cuda()

    def step():
        fs.clip_grad_norm(grads, 0.05, out=out, norm=norm, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        for g in grads:
            g.mul_(1.5)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        got = [norm.clone(), *[o.clone() for o in out]]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, [norm, *out])), i


def test_refusals():
    a, b = torch.ones(4).cuda(), torch.ones(4).cuda()
    with pytest.raises(ValueError):
        fs.clip_grad_norm([a, a], 1.0)            # written twice
    base = torch.ones(10).cuda()
    with pytest.raises(ValueError):
        fs.clip_grad_norm([base[:6], base[4:]], 1.0)
    with pytest.raises(ValueError):
        fs.clip_grad_norm([a, b], 1.0, out=[b, torch.empty_like(b)])   # out[0] is grads[1]
    with pytest.raises(ValueError):
        fs.clip_grad_norm([base[:4], base[6:]], 1.0, out=[base[3:7], torch.empty(4).cuda()])
    fs.clip_grad_norm([a, a], 9.0, out=[torch.empty_like(a), torch.empty_like(a)])  # read twice: fine
    with pytest.raises(ValueError):
        fs.clip_grad_norm([a, b], 1.0, out=[a])
    with pytest.raises(ValueError):
        fs.clip_grad_norm([a], 1.0, out=[torch.ones(5).cuda()])
    with pytest.raises(ValueError):
        fs.clip_grad_norm([torch.ones(4, 4).cuda().t()], 1.0)
    with pytest.raises(TypeError):
        fs.clip_grad_norm([a.double()], 1.0)
    with pytest.raises(fs.FlashSampleError):
        fs.clip_grad_norm([a], -1.0)
    assert (a == 1).all()
