"""The fp64 reference of the cross entropy against torch's own in fp64 and
against differences (CPU), so that the GPU tests rest on a checked formula."""
import pytest
import torch

import head_ref

F64 = torch.float64


def make(B, D, V, seed=0):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(B, D, generator=g, dtype=F64)
    W = torch.randn(V, D, generator=g, dtype=F64)
    t = torch.randint(0, V, (B,), generator=g).to(torch.int32)
    t[1::3] = -100
    return h, W, t


@pytest.mark.parametrize("smoothing", [0.0, 0.1, 1.0])
@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_against_torch(smoothing, reduction):
    h, W, t = make(7, 5, 11)
    h.requires_grad_(True)
    W.requires_grad_(True)
    loss = torch.nn.functional.cross_entropy(h @ W.T, t.long(), label_smoothing=smoothing,
                                             reduction=reduction, ignore_index=-100)
    loss.backward()
    r = head_ref.cross_entropy(h.detach(), W.detach(), t, smoothing, 0.0, reduction)
    assert abs(float(r["stats"][0]) - float(loss.detach())) < 1e-12
    assert (r["grad_h"] - h.grad).abs().max() < 1e-12
    assert (r["grad_W"] - W.grad).abs().max() < 1e-12


@pytest.mark.parametrize("smoothing,z_loss", [(0.0, 0.3), (0.2, 0.05)])
def test_gradient_against_differences(smoothing, z_loss):
    h, W, t = make(4, 3, 5, seed=1)
    kw = dict(label_smoothing=smoothing, z_loss=z_loss, reduction="mean", grad_scale=1.0)
    r = head_ref.cross_entropy(h, W, t, **kw)
    eps = 1e-6
    for x, g in ((h, r["grad_h"]), (W, r["grad_W"])):
        for i in range(x.numel()):
            at = x.view(-1)
            keep = float(at[i])
            at[i] = keep + eps
            up = float(head_ref.cross_entropy(h, W, t, **kw)["stats"][0])
            at[i] = keep - eps
            down = float(head_ref.cross_entropy(h, W, t, **kw)["stats"][0])
            at[i] = keep
            assert abs((up - down) / (2 * eps) - float(g.reshape(-1)[i])) < 1e-8


def test_bounds_cover_the_gradients():
    h, W, t = make(6, 4, 9, seed=2)
    r = head_ref.cross_entropy(h, W, t, 0.1, 0.02, "sum", -3.0)
    assert (r["grad_h"].abs() <= r["bound_h"] + 1e-12).all()
    assert (r["grad_W"].abs() <= r["bound_W"] + 1e-12).all()
