"""Plain fp64 references of the LM head's cross entropy (test infrastructure):
written from the definition; they share no code with the library."""
import math

import torch

F64 = torch.float64


def cross_entropy(h, W, targets, label_smoothing=0.0, z_loss=0.0, reduction="mean", grad_scale=1.0):
    """dict of stats [3], losses [B], grad_h, grad_W and, for the tolerances, lse
    [B], nll [B] and the sums of absolute terms bound_h and bound_W that a
    rounding of dz is relative to.  On the tensors' device."""
    B, V = h.shape[0], W.shape[0]
    dev = h.device
    on = targets.long() >= 0
    h64 = torch.where(on[:, None], h.to(F64), torch.zeros((), dtype=F64, device=dev))
    W64 = W.to(F64)
    z = h64 @ W64.T
    lse = torch.logsumexp(z, dim=1)
    y = targets.long()
    here = on & (y < V)
    hot = torch.zeros(B, V, dtype=torch.bool, device=dev)
    hot[here, y[here]] = True
    rest = torch.logsumexp(z.masked_fill(hot, -math.inf), dim=1)
    zt = (z.masked_fill(~hot, 0.0)).sum(dim=1)
    x = torch.where(here, rest - zt, torch.full_like(rest, math.inf))
    nll = torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-x.abs()))
    s, lam = label_smoothing, z_loss
    losses = (1 - s) * nll if s < 1 else torch.zeros_like(nll)
    if s > 0:
        losses = losses + s * (lse - z.mean(dim=1))
    if lam > 0:
        losses = losses + lam * lse ** 2
    losses = torch.where(on, losses, torch.zeros_like(losses))
    n = int(on.sum())
    share = 1.0 / max(n, 1) if reduction == "mean" else 1.0

    def mean(v):
        return float(v[on].sum()) / max(n, 1)

    stats = torch.tensor([float(losses.sum()) * share, mean(nll), mean(lse ** 2)], dtype=F64)
    u = torch.where(on, torch.full((B,), grad_scale * share, dtype=F64, device=dev),
                    torch.zeros((), dtype=F64, device=dev))
    lift = (1 + 2 * lam * lse)[:, None]
    p = torch.exp(z - lse[:, None])
    nll = torch.where(on, nll, torch.zeros_like(nll))
    own = torch.expm1(-nll) + 2 * lam * lse * torch.exp(-nll) + s - s / V
    size = lift.abs() * p + s / V
    size = torch.where(hot, (-torch.expm1(-nll) + 2 * lam * lse.abs() * torch.exp(-nll) + s)[:, None], size)
    dz = torch.where(hot, own[:, None], lift * p - s / V) * u[:, None]
    size = size * u.abs()[:, None]
    return dict(stats=stats, losses=losses, lse=lse, nll=nll, grad_h=dz @ W64, grad_W=dz.T @ h64,
                bound_h=size @ W64.abs(), bound_W=size.T @ h64.abs())
