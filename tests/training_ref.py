"""Plain fp64 references of the training operators (test infrastructure).

Written from the definitions, sequence by sequence and with torch's autograd
for the losses' gradients, on the CPU; they share no code with the library.
"""
import math

import torch

F64 = torch.float64


def inv_temperature(T, B):
    """fp32(1/T) per row; rows whose temperature is not positive: 1."""
    if T is None:
        return torch.ones(B, dtype=F64)
    out = [float(torch.tensor(1.0) / t) if float(t) > 0 else 1.0 for t in T.float().cpu()]
    return torch.tensor(out, dtype=F64)


def scaled_logits(h, W, T):
    return (h.cpu().to(F64) @ W.cpu().to(F64).T) * inv_temperature(T, h.shape[0])[:, None]


def logprobs(h, W, T, ids, off):
    """(logprob, lse) of each row."""
    t = scaled_logits(h, W, T)
    lp, lse = [], torch.logsumexp(t, dim=1)
    for b, i in enumerate(ids.tolist()):
        if i < 0:
            lp.append(0.0)
        elif not off <= i < off + W.shape[0]:
            lp.append(-math.inf)
        else:
            rest = t[b].clone()
            rest[i - off] = -math.inf
            x = float(torch.logsumexp(rest, dim=0) - t[b, i - off])
            lp.append(-(max(x, 0.0) + math.log1p(math.exp(-abs(x)))))
    return torch.tensor(lp, dtype=F64), lse


def logit_tolerance(h, W, T):
    """Largest rounding error of a scaled logit, fp32 accumulation: D additions
    whose partial sums have the size of a random walk, |sum| <= sqrt(D) s for
    terms of root mean square s, each rounded by 2^-24 of it, independently:
    2^-24 D s = 2^-24 sqrt(D) |h . W| (elementwise product's norm); four of
    those, and 2^-23 for the two roundings of the scaling."""
    h64, W64 = h.cpu().to(F64), W.cpu().to(F64)
    beta = inv_temperature(T, h.shape[0])
    norm = ((h64 ** 2) @ (W64 ** 2).T).sqrt() * beta[:, None]
    big = scaled_logits(h, W, T).abs()
    return float((4 * 2.0 ** -24 * math.sqrt(h.shape[1]) * norm + 2.0 ** -23 * big).max())


def logprobs_backward(h, W, T, ids, off, lp, lse, g):
    """(grad_h, grad_W, bound_h, bound_W): bounds are sums of absolute terms
    |dz| |W| and |dz|^T |h|, what the rounding of dz is relative to."""
    B, V = h.shape[0], W.shape[0]
    t = scaled_logits(h, W, T)
    beta = inv_temperature(T, B)
    dz = torch.zeros(B, V, dtype=F64)
    hz = torch.zeros(h.shape, dtype=F64)
    for b, i in enumerate(ids.tolist()):
        if i < 0:
            continue
        hz[b] = h[b].cpu().to(F64)
        row = -torch.exp(t[b] - float(lse[b]))
        if off <= i < off + V:
            row[i - off] = -math.expm1(float(lp[b]))
        dz[b] = row * float(g[b]) * beta[b]
    W64 = W.cpu().to(F64)
    return dz @ W64, dz.T @ hz, dz.abs() @ W64.abs(), dz.abs().T @ hz.abs()


def _keep(cu, mask, s, N):
    a, b = cu[s], cu[s + 1]
    m = torch.ones(N, dtype=torch.bool) if mask is None else mask.cpu().bool()
    return [t for t in range(a, b) if m[t]]


def policy(lp, old, adv, cu, ref=None, mask=None, per_token=False, clip_low=0.2, clip_high=0.2,
           dual_clip=0.0, kl_coef=0.0, kl="k3", reduction="token"):
    """(stats [4], grad [N]); grad by autograd of the loss (torch's min and
    clamp pass the gradient of the branch they take)."""
    cu = cu.tolist()
    N, S = lp.shape[0], len(cu) - 1
    x = lp.cpu().to(F64).clone().requires_grad_(True)
    old, adv = old.cpu().to(F64), adv.cpu().to(F64)
    ref = None if ref is None else ref.cpu().to(F64)
    surr_seq, kl_seq, counts, hit = [], [], [], 0
    for s in range(S):
        k = _keep(cu, mask, s, N)
        if not k:
            continue
        A = adv[k] if per_token else adv[s].expand(len(k))
        r = torch.exp(x[k] - old[k])
        rA, cA = r * A, torch.clamp(r, 1 - clip_low, 1 + clip_high) * A
        clipped = rA > cA
        take = torch.where(clipped, cA.detach(), rA)
        if dual_clip > 0:
            cap = (A < 0) & (take < dual_clip * A)
            take = torch.where(cap, (dual_clip * A).detach(), take)
            clipped = clipped | cap
        hit += int(clipped.sum())
        surr_seq.append(-take.sum())
        counts.append(len(k))
        if ref is None:
            kl_seq.append(torch.zeros((), dtype=F64))
        else:
            q = ref[k] - x[k]
            kl_seq.append({"k1": -q, "k2": q * q / 2, "k3": torch.expm1(q) - q}[kl].sum())
    if not counts:
        return torch.zeros(4, dtype=F64), torch.zeros(N, dtype=F64)
    if reduction == "token":
        w = [1.0 / sum(counts)] * len(counts)
    else:
        w = [1.0 / (n * len(counts)) for n in counts]
    surr = sum(v * a for v, a in zip(surr_seq, w))
    klm = sum(v * a for v, a in zip(kl_seq, w))
    loss = surr + kl_coef * klm
    loss.backward()
    stats = torch.tensor([float(loss.detach()), float(surr.detach()), float(klm.detach()), hit / sum(counts)], dtype=F64)
    return stats, x.grad.clone()


def preference(lp, cu, ref=None, mask=None, kind="sigmoid", beta=0.1, margin=0.0,
               label_smoothing=0.0, length_normalised=False):
    """(stats [3], rewards [2P], grad [N])."""
    cu = cu.tolist()
    N, P = lp.shape[0], (len(cu) - 1) // 2
    x = lp.cpu().to(F64).clone().requires_grad_(True)
    base = torch.zeros(N, dtype=F64) if ref is None else ref.cpu().to(F64)
    score, size = [], []
    for s in range(2 * P):
        k = _keep(cu, mask, s, N)
        v = (x[k] - base[k]).sum() if k else torch.zeros((), dtype=F64)
        score.append(v / len(k) if length_normalised and k else v)
        size.append(len(k))
    live = [p for p in range(P) if size[p] and size[P + p]]
    rewards = torch.tensor([beta * float(v.detach()) for v in score], dtype=F64)
    if not live:
        return torch.zeros(3, dtype=F64), rewards, torch.zeros(N, dtype=F64)
    loss = torch.zeros((), dtype=F64)
    acc = gap = 0.0
    for p in live:
        d = score[p] - score[P + p]
        u = beta * d - margin
        if kind == "ipo":
            one = (d - 0.5 / beta) ** 2
        elif kind == "hinge":
            one = torch.clamp(1 - u, min=0.0)
        else:
            ls = torch.nn.functional.logsigmoid   # (its gradient is finite at any margin)
            one = -(1 - label_smoothing) * ls(u) - label_smoothing * ls(-u)
        loss = loss + one / len(live)
        acc += (float(d.detach()) > 0) / len(live)
        gap += beta * float(d.detach()) / len(live)
    loss.backward()
    return (torch.tensor([float(loss.detach()), acc, gap], dtype=F64), rewards, x.grad.clone())


def clip(grads, max_norm):
    """(norm, scaled tensors in fp64)."""
    sq = math.fsum(float((g.cpu().to(F64) ** 2).sum()) for g in grads)
    norm = math.sqrt(sq) if math.isfinite(sq) else sq
    c = 1.0
    if math.isfinite(norm):
        c = min(1.0, max_norm / (norm + 1e-6))
    return norm, [g.cpu().to(F64) * c for g in grads]
